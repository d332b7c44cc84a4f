// lm_api.cpp -- host side of the operators on token IDs: argument checks and
// launches.
#include <hip/hip_runtime.h>

#include "lm_internal.h"

using namespace bpe;

namespace {

bool type_ok(int t) { return t == BPE_F32 || t == BPE_BF16 || t == BPE_F16; }

bool table_ok(int64_t n_rows, int64_t width) {
  return n_rows >= 1 && n_rows <= BPE_MAX_ROWS && width >= 1 && width <= BPE_MAX_WIDTH;
}

// The sort's part of a gradient's arguments.
void sort_args(GradArgs *a, const GradLayout &L, uint8_t *ws) {
  a->key[0] = (int32_t *)(ws + L.key0);
  a->key[1] = (int32_t *)(ws + L.key1);
  a->pos[0] = (int32_t *)(ws + L.pos0);
  a->pos[1] = (int32_t *)(ws + L.pos1);
  a->counts = (int32_t *)(ws + L.counts);
  a->sort_tiles = L.sort_tiles;
  a->sort_steps = L.sort_steps;
  a->passes = L.passes;
  a->bits = L.bits;
}

// Whether rows of `stride` elements can be addressed in 64 bits.
bool stride_ok(int64_t stride, int64_t width) {
  return stride >= width && stride <= ((int64_t)1 << 32);
}

bool distill_ok(int student_type, int64_t n_rows, int64_t vocab, int64_t student_stride,
                int64_t ids_stride, int teacher_type, int64_t teacher_stride, int64_t top,
                float temperature) {
  return type_ok(student_type) && type_ok(teacher_type) && n_rows >= 0 &&
         launch_fits(n_rows, kDistillThreads) && vocab >= 1 && vocab <= BPE_MAX_ROWS &&
         stride_ok(student_stride, vocab) && top >= 0 && top <= BPE_MAX_TOP &&
         stride_ok(ids_stride, top) && stride_ok(teacher_stride, top) && temperature >= 0x1p-20f &&
         temperature <= 0x1p20f;
}

}  // namespace

extern "C" {

size_t bpe_embed_workspace_bytes(int64_t n_ids, int64_t n_rows, int64_t width, int weight_type,
                                 int out_type) {
  if (!type_ok(weight_type) || !type_ok(out_type) || n_ids <= 0 || n_ids > BPE_MAX_IDS ||
      !table_ok(n_rows, width) || !embed_fits(n_ids, width, out_type) ||
      !by_sorted_ids(n_ids, n_rows, width, weight_type, out_type))
    return 0;
  return grad_layout(n_ids, n_rows, width).touched;  // what the sort needs comes first
}

int bpe_embed(const void *d_weight, int weight_type, int64_t n_rows, int64_t width,
              int64_t weight_stride, const int32_t *d_ids, int64_t n_ids, float scale,
              int32_t pad_id, void *d_out, int out_type, int64_t out_stride, void *d_workspace,
              size_t workspace_bytes, int32_t *d_status, void *hip_stream) {
  if (!type_ok(weight_type) || !type_ok(out_type) || !table_ok(n_rows, width) || n_ids < 0 ||
      n_ids > BPE_MAX_IDS || !stride_ok(weight_stride, width) || !stride_ok(out_stride, width) ||
      pad_id < -1 || !d_status || (n_ids > 0 && (!d_weight || !d_ids || !d_out)))
    return BPE_EINVAL;
  if (n_ids == 0) return BPE_OK;
  if (!embed_fits(n_ids, width, out_type)) return BPE_EINVAL;
  EmbedArgs a = {};
  a.weight = d_weight;
  a.ids = d_ids;
  a.out = d_out;
  a.status = d_status;
  a.n_rows = n_rows;
  a.n_ids = n_ids;
  a.w_stride = weight_stride;
  a.o_stride = out_stride;
  a.width = (int32_t)width;
  a.pad_id = pad_id;
  a.scale = scale;
  GradArgs s = {};
  const size_t need = bpe_embed_workspace_bytes(n_ids, n_rows, width, weight_type, out_type);
  if (need > 0) {
    if (workspace_bytes < need) return BPE_EWORKSPACE;
    if (!d_workspace || ((uintptr_t)d_workspace & 15)) return BPE_EINVAL;
    sort_args(&s, grad_layout(n_ids, n_rows, width), (uint8_t *)d_workspace);
    s.ids = d_ids;
    s.n_ids = n_ids;
    s.n_rows = n_rows;
    s.pad_id = pad_id;
    s.status = d_status;
    a.key = s.key[(s.passes - 1) & 1];
    a.pos = s.pos[(s.passes - 1) & 1];
  }
  return launch_embed(a, need > 0 ? &s : nullptr, weight_type, out_type,
                      (hipStream_t)hip_stream) == hipSuccess
             ? BPE_OK
             : BPE_EHIP;
}

size_t bpe_embed_grad_workspace_bytes(int64_t n_ids, int64_t n_rows, int64_t width) {
  if (n_ids <= kGradDirect || n_ids > BPE_MAX_IDS || !table_ok(n_rows, width) ||
      !grad_fits(n_ids, n_rows, width))
    return 0;
  return grad_layout(n_ids, n_rows, width).total;
}

int bpe_embed_grad(const void *d_grad, int grad_type, int64_t grad_stride, const int32_t *d_ids,
                   int64_t n_ids, int64_t n_rows, int64_t width, float scale, int32_t pad_id,
                   int accumulate, void *d_out, int out_type, int64_t out_stride,
                   void *d_workspace, size_t workspace_bytes, int32_t *d_status,
                   void *hip_stream) {
  if (!type_ok(grad_type) || !type_ok(out_type) || !table_ok(n_rows, width) || n_ids < 0 ||
      n_ids > BPE_MAX_IDS || !stride_ok(grad_stride, width) || !stride_ok(out_stride, width) ||
      pad_id < -1 || !d_status || !d_out ||
      (n_ids > 0 && (!d_grad || !d_ids || (n_ids > kGradDirect && !d_workspace))))
    return BPE_EINVAL;
  GradArgs a = {};
  a.grad = d_grad;
  a.ids = d_ids;
  a.out = d_out;
  a.status = d_status;
  a.n_rows = n_rows;
  a.n_ids = n_ids;
  a.g_stride = grad_stride;
  a.o_stride = out_stride;
  a.width = (int32_t)width;
  a.pad_id = pad_id;
  a.scale = scale;
  a.accumulate = accumulate != 0;
  if (n_ids > kGradDirect) {
    if (!grad_fits(n_ids, n_rows, width)) return BPE_EINVAL;
    const GradLayout L = grad_layout(n_ids, n_rows, width);
    if (workspace_bytes < L.total) return BPE_EWORKSPACE;
    if ((uintptr_t)d_workspace & 15) return BPE_EINVAL;
    uint8_t *ws = (uint8_t *)d_workspace;
    sort_args(&a, L, ws);
    a.touched = ws + L.touched;
    a.part = (float *)(ws + L.part);
    a.tile = L.tile;
    a.tiles = L.tiles;
  }
  return launch_embed_grad(a, grad_type, out_type, (hipStream_t)hip_stream) == hipSuccess
             ? BPE_OK
             : BPE_EHIP;
}

int bpe_process_logits(const bpe_logits_args *args, void *hip_stream) {
  if (!args) return BPE_EINVAL;
  const bpe_logits_args &a = *args;
  if (!type_ok(a.logits_type) || !type_ok(a.out_type) || a.rows < 0 || a.rows > BPE_MAX_IDS ||
      a.vocab < 0 || a.vocab > BPE_MAX_ROWS || !stride_ok(a.logits_stride, a.vocab) ||
      !stride_ok(a.out_stride, a.vocab) || !a.status)
    return BPE_EINVAL;
  const bool any = a.rows > 0 && a.vocab > 0;
  if (any && (!a.logits || !a.out)) return BPE_EINVAL;
  if (any && a.out == a.logits &&
      (a.out_type != a.logits_type || a.out_stride != a.logits_stride))
    return BPE_EINVAL;
  // each list is there or left out as a whole; one without entries needs no
  // entries' pointer
  if (a.n_prompt < 0 || a.n_bias < 0 || a.n_masks < 0 || a.n_masks > INT32_MAX ||
      a.made_width < 0)
    return BPE_EINVAL;
  if (a.prompt_off ? a.n_prompt > 0 && !a.prompt_ids : a.prompt_ids != nullptr) return BPE_EINVAL;
  if (a.made_len ? a.made_width > 0 && !a.made_ids : a.made_ids != nullptr) return BPE_EINVAL;
  if (a.bias_off ? a.n_bias > 0 && (!a.bias_ids || !a.bias_values)
                 : a.bias_ids || a.bias_values)
    return BPE_EINVAL;
  if (a.mask_row ? a.n_masks > 0 && !a.mask : a.mask != nullptr) return BPE_EINVAL;
  // a count is kept in 21 bits
  if (a.made_ids && (a.made_width >= (1 << 21) || !stride_ok(a.made_stride, a.made_width)))
    return BPE_EINVAL;
  if (a.mask && !stride_ok(a.mask_stride, (a.vocab + 31) / 32)) return BPE_EINVAL;
  if (!any) return BPE_OK;
  if (!logits_fit(a)) return BPE_EINVAL;
  return launch_logits(a, (hipStream_t)hip_stream) == hipSuccess ? BPE_OK : BPE_EHIP;
}

size_t bpe_block_tables_workspace_bytes(int64_t n_requests, int64_t n_new) {
  if (n_requests <= kBlockFused || n_new < 0) return 0;
  return (size_t)n_requests * 8 + kBlockGroups * 8 +
         (size_t)((n_new + kBlockChunk - 1) / kBlockChunk) * 4;
}

int bpe_block_tables(const int64_t *d_new_off, int64_t n_requests, int64_t n_new,
                     const int32_t *d_cached, const int32_t *d_free_blocks, int64_t n_free,
                     int32_t *d_table, int64_t table_width, int64_t table_stride,
                     int32_t block_size, int64_t *d_slots, int32_t *d_positions,
                     int32_t *d_lengths, int64_t *d_used, void *d_workspace,
                     size_t workspace_bytes, int32_t *d_status, void *hip_stream) {
  if (n_requests < 0 || n_requests > BPE_MAX_IDS || n_new < 0 || n_new > kBlockMaxNew ||
      n_free < 0 || block_size < 1 || table_width < 0 || table_width > INT32_MAX ||
      !stride_ok(table_stride, table_width) || !d_status || !d_used ||
      (n_new > 0 && n_requests == 0) || (n_free > 0 && !d_free_blocks))
    return BPE_EINVAL;
  if (n_requests > 0 && (!d_new_off || !d_cached || !d_lengths ||
                         (n_requests > kBlockFused && !d_workspace) ||
                         (table_width > 0 && !d_table)))
    return BPE_EINVAL;
  if (n_new > 0 && (!d_slots || !d_positions)) return BPE_EINVAL;
  if (workspace_bytes < bpe_block_tables_workspace_bytes(n_requests, n_new)) return BPE_EWORKSPACE;
  BlockArgs a = {};
  a.off = d_new_off;
  a.R = n_requests;
  a.T = n_new;
  a.cached = d_cached;
  a.free_blocks = d_free_blocks;
  a.n_free = n_free;
  a.table = d_table;
  a.width = table_width;
  a.stride = table_stride;
  a.bs = block_size;
  block_divisor(block_size, &a.magic, &a.shift);
  a.slots = d_slots;
  a.positions = d_positions;
  a.lengths = d_lengths;
  a.used = d_used;
  a.status = d_status;
  if (n_requests > kBlockFused) {
    if ((uintptr_t)d_workspace & 7) return BPE_EINVAL;
    a.first = (int64_t *)d_workspace;
    a.gsum = a.first + n_requests;
    a.chunk_req = (int32_t *)(a.gsum + kBlockGroups);
  }
  a.group_log2 = 10;
  while (((n_requests - 1) >> a.group_log2) + 1 > kBlockGroups) ++a.group_log2;
  return launch_blocks(a, (hipStream_t)hip_stream) == hipSuccess ? BPE_OK : BPE_EHIP;
}

int bpe_cache_write(const bpe_cache *cache, const void *d_x, int x_type, int64_t n,
                    int64_t token_stride, int64_t head_stride, const int64_t *d_slots,
                    int32_t *d_status, void *hip_stream) {
  if (!cache || !type_ok(x_type) || !cache_ok(*cache) ||
      !cache_tokens_ok(*cache, n, token_stride, head_stride) || !d_status ||
      (n > 0 && (!d_x || !d_slots)))
    return BPE_EINVAL;
  if (n == 0) return BPE_OK;
  CacheArgs a = {};
  a.c = *cache;
  a.n = n;
  a.t_stride = token_stride;
  a.h_stride = head_stride;
  a.status = d_status;
  a.x = d_x;
  a.slots = d_slots;
  cache_shape(&a, true, x_type);
  if (!cache_fits(a)) return BPE_EINVAL;
  return launch_cache_write(a, x_type, (hipStream_t)hip_stream) == hipSuccess ? BPE_OK : BPE_EHIP;
}

int bpe_cache_read(const bpe_cache *cache, const int32_t *d_table, int64_t n_requests,
                   int64_t table_width, int64_t table_stride, int32_t block_size,
                   const int64_t *d_off, const int32_t *d_start, int64_t n, void *d_out,
                   int out_type, int64_t token_stride, int64_t head_stride, int32_t *d_status,
                   void *hip_stream) {
  if (!cache || !type_ok(out_type) || !cache_ok(*cache) ||
      !cache_tokens_ok(*cache, n, token_stride, head_stride) || n_requests < 0 ||
      n_requests > BPE_MAX_IDS || table_width < 0 || table_width > INT32_MAX ||
      !stride_ok(table_stride, table_width) || block_size < 1 || !d_status || (n > 0 && !d_out) ||
      (n_requests > 0 && (!d_off || (table_width > 0 && !d_table))))
    return BPE_EINVAL;
  if (n == 0 || n_requests == 0) return BPE_OK;
  CacheArgs a = {};
  a.c = *cache;
  a.n = n;
  a.t_stride = token_stride;
  a.h_stride = head_stride;
  a.status = d_status;
  a.out = d_out;
  a.table = d_table;
  a.start = d_start;
  a.off = d_off;
  a.R = n_requests;
  a.width = table_width;
  a.stride = table_stride;
  a.bs = divisor(block_size);
  cache_shape(&a, false, out_type);
  if (!cache_fits(a)) return BPE_EINVAL;
  return launch_cache_read(a, out_type, (hipStream_t)hip_stream) == hipSuccess ? BPE_OK : BPE_EHIP;
}

size_t bpe_verify_drafts_workspace_bytes(int64_t n_requests, int64_t vocab) {
  if (n_requests <= 0 || n_requests >= (1 << 20) || verify_alone(n_requests, vocab) || vocab > BPE_MAX_ROWS)
    return 0;
  return (size_t)n_requests * (verify_regions(vocab) * 8 + 4);
}

int bpe_verify_drafts(const void *d_target, int prob_type, int64_t n_rows, int64_t vocab,
                      int64_t target_stride, const void *d_draft, int64_t draft_stride,
                      const int32_t *d_draft_ids, const int64_t *d_row_off, int64_t n_requests,
                      const float *d_accept, const float *d_sample, int32_t *d_tokens,
                      int32_t *d_counts, void *d_workspace, size_t workspace_bytes,
                      int32_t *d_status, void *hip_stream) {
  if (!type_ok(prob_type) || n_rows < 0 || n_rows > BPE_MAX_IDS || vocab < 1 ||
      vocab > BPE_MAX_ROWS || !stride_ok(target_stride, vocab) ||
      (d_draft && !stride_ok(draft_stride, vocab)) || n_requests < 0 ||
      n_requests >= (1 << 20) || !d_status ||
      (n_rows > 0 && (!d_target || !d_draft_ids || !d_accept || !d_tokens)) ||
      (n_requests > 0 && (!d_row_off || !d_sample || !d_counts)))
    return BPE_EINVAL;
  if (n_requests == 0) return BPE_OK;
  VerifyArgs a = {};
  if (!verify_alone(n_requests, vocab)) {
    if (workspace_bytes < bpe_verify_drafts_workspace_bytes(n_requests, vocab)) return BPE_EWORKSPACE;
    if (!d_workspace || ((uintptr_t)d_workspace & 7)) return BPE_EINVAL;
    a.sums = (double *)d_workspace;
    a.rows = (int32_t *)(a.sums + n_requests * verify_regions(vocab));
    if (!launch_fits(verify_workgroups(n_requests, vocab), kVerifyThreads)) return BPE_EINVAL;
  }
  a.regions = verify_regions(vocab);
  a.tiles = verify_tiles(vocab);
  a.target = d_target;
  a.draft = d_draft;
  a.n_rows = n_rows;
  a.vocab = vocab;
  a.t_stride = target_stride;
  a.d_stride = draft_stride;
  a.ids = d_draft_ids;
  a.off = d_row_off;
  a.R = n_requests;
  a.accept = d_accept;
  a.sample = d_sample;
  a.tokens = d_tokens;
  a.counts = d_counts;
  a.status = d_status;
  return launch_verify(a, prob_type, (hipStream_t)hip_stream) == hipSuccess ? BPE_OK : BPE_EHIP;
}

int bpe_distill(const void *d_student, int student_type, int64_t n_rows, int64_t vocab,
                int64_t student_stride, const int32_t *d_ids, int64_t ids_stride,
                const void *d_teacher, int teacher_type, int64_t teacher_stride, int64_t top,
                float temperature, float *d_losses, float *d_stats, int32_t *d_status,
                void *hip_stream) {
  if (!distill_ok(student_type, n_rows, vocab, student_stride, ids_stride, teacher_type,
                  teacher_stride, top, temperature) ||
      !d_status || (n_rows > 0 && (!d_student || !d_losses || !d_stats || (top > 0 && (!d_ids || !d_teacher)))))
    return BPE_EINVAL;
  if (n_rows == 0) return BPE_OK;
  DistillArgs a = {};
  a.student = d_student;
  a.teacher = d_teacher;
  a.rows = n_rows;
  a.vocab = vocab;
  a.s_stride = student_stride;
  a.t_stride = teacher_stride;
  a.ids = d_ids;
  a.i_stride = ids_stride;
  a.top = (int32_t)top;
  a.t_type = teacher_type;
  a.temperature = temperature;
  a.losses = d_losses;
  a.stats = d_stats;
  a.status = d_status;
  return launch_distill(a, student_type, (hipStream_t)hip_stream) == hipSuccess
             ? BPE_OK
             : BPE_EHIP;
}

int bpe_distill_grad(const void *d_student, int student_type, int64_t n_rows, int64_t vocab,
                     int64_t student_stride, const int32_t *d_ids, int64_t ids_stride,
                     const void *d_teacher, int teacher_type, int64_t teacher_stride, int64_t top,
                     const float *d_stats, const float *d_dloss, float temperature, void *d_grad,
                     int grad_type, int64_t grad_stride, int32_t *d_status, void *hip_stream) {
  if (!distill_ok(student_type, n_rows, vocab, student_stride, ids_stride, teacher_type,
                  teacher_stride, top, temperature) ||
      !type_ok(grad_type) || !stride_ok(grad_stride, vocab) || !d_status ||
      (n_rows > 0 && (!d_student || !d_stats || !d_dloss || !d_grad || (top > 0 && (!d_ids || !d_teacher)))))
    return BPE_EINVAL;
  if (d_grad && d_grad == d_student && (grad_type != student_type || grad_stride != student_stride))
    return BPE_EINVAL;
  if (n_rows == 0) return BPE_OK;
  if (!distill_grad_fits(n_rows, vocab)) return BPE_EINVAL;
  DistillArgs a = {};
  a.student = d_student;
  a.teacher = d_teacher;
  a.rows = n_rows;
  a.vocab = vocab;
  a.s_stride = student_stride;
  a.t_stride = teacher_stride;
  a.ids = d_ids;
  a.i_stride = ids_stride;
  a.top = (int32_t)top;
  a.t_type = teacher_type;
  a.temperature = temperature;
  a.in_stats = d_stats;
  a.dloss = d_dloss;
  a.grad = d_grad;
  a.g_stride = grad_stride;
  a.status = d_status;
  return launch_distill_grad(a, student_type, grad_type, (hipStream_t)hip_stream) == hipSuccess
             ? BPE_OK
             : BPE_EHIP;
}

}  // extern "C"
