// C ABI of the paged calls: argument checks, kernel selection, launches.  See
// include/mtla.h for the contract of every entry point.
#include <math.h>
#include <string.h>

#include "paged.cuh"

namespace {

using namespace mtla;

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
size_t elem(int dtype) { return dtype == MTLA_BF16 ? 2 : 4; }
bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + nb && y < x + na;
}
mtla_status from_cuda(cudaError_t e) { return e == cudaSuccess ? MTLA_OK : MTLA_ERR_CUDA; }

mtla_status chunk_args(int32_t B, const mtla_chunk* c, ChunkDev* d) {
  if (B < 0 || !c || c->N < 0 || !c->tok_start || !c->t_prev) return MTLA_ERR_INVALID_ARG;
  if (!aligned(c->tok_start, 4) || !aligned(c->tok_count, 4) || !aligned(c->t_prev, 4)) return MTLA_ERR_INVALID_ARG;
  d->B = B;
  d->N = c->N;
  d->tok_start = c->tok_start;
  d->tok_count = c->tok_count;
  d->t_prev = c->t_prev;
  return MTLA_OK;
}

mtla_status cache_args(const mtla_dims* dims, const mtla_paged_cache* c, PagesDev* d) {
  if (!c || !c->pages || !c->block_table || !aligned(c->pages, 16) || !aligned(c->block_table, 4))
    return MTLA_ERR_INVALID_ARG;
  if (c->page_rows < 8 || c->page_rows % 8 || c->num_pages < 1 || c->table_pages < 1) return MTLA_ERR_INVALID_ARG;
  if (c->num_pages > ((int64_t(1) << 31) - 1) / c->page_rows) return MTLA_ERR_INVALID_ARG;
  if (c->row_stride < dims->r + dims->d_R || c->row_stride >= (int64_t(1) << 31) ||
      (c->row_stride * (int64_t)elem(dims->dtype)) % 16)
    return MTLA_ERR_INVALID_ARG;
  d->pages = c->pages;
  d->num_pages = c->num_pages;
  d->row_stride = c->row_stride;
  d->table = c->block_table;
  d->page_rows = c->page_rows;
  d->table_pages = c->table_pages;
  d->div_rows = fast_div((uint32_t)c->page_rows);
  return MTLA_OK;
}

// The attention's kernel, the blocks of its persistent grid and the rows of
// its M tiles.  The tensor-core kernel takes the widths its operand planes and
// TMEM columns are laid out for; its one block an SM needs no query.
struct AttnShape {
  bool tc;
  int grid, rows;
};
AttnShape attn_shape(const mtla_dims* d) {
  AttnShape s = {false, 0, 0};
  const int sms = current_device_sms();
  if (sms <= 0) return s;
  s.tc = d->dtype == MTLA_BF16 && d->r == 256 && d->d_R == 32;
  s.grid = s.tc ? sms : paged_simt_grid(d->r, d->d_R, d->dtype, sms);
  s.rows = s.tc ? PTC_ROWS : PSM;
  return s;
}

// Rows of width 288 in bf16 (or the 256 latents of a query) as planes of 32
// elements, boxes of 8 rows: a box lands as one operand group, plane by plane.
bool row_groups_map(CUtensorMap* m, const void* base, int64_t rows, int64_t stride_bytes, int planes) {
  const cuuint64_t d[3] = {32, (cuuint64_t)rows, (cuuint64_t)planes}, st[2] = {(cuuint64_t)stride_bytes, 64};
  const cuuint32_t box[3] = {32, 8, (cuuint32_t)planes};
  return encode_bf16_tiled_map(m, base, 3, d, st, box, CU_TENSOR_MAP_SWIZZLE_64B);
}
bool paged_maps(PagedAttnMaps* m, const PagedAttnArgs& a) {
  const int64_t rows = (int64_t)a.c.N * a.H;
  const cuuint64_t d[2] = {32, (cuuint64_t)rows}, st[1] = {64};
  const cuuint32_t box[2] = {32, 8};
  return row_groups_map(&m->q, a.q_abs, rows, 512, 8) &&
         encode_bf16_tiled_map(&m->qr, a.q_rope, 2, d, st, box, CU_TENSOR_MAP_SWIZZLE_64B) &&
         row_groups_map(&m->own, a.row_state, a.c.N, 576, 9) &&
         row_groups_map(&m->cache, a.p.pages, a.p.num_pages * a.p.page_rows, a.p.row_stride * 2, 9);
}

// The angles of one position; a thread keeps the last ones (16 long powers cost
// as much as the launch).
void rope_table(double base, int d_R, RopeTable* t) {
  struct Last {
    double base = 0.0;
    int d_R = 0;
    RopeTable t;
  };
  thread_local Last last;
  if (last.base != base || last.d_R != d_R) {
    for (int k = 0; k < d_R / 2; ++k) {
      const long double turn = powl((long double)base, -2.0L * k / d_R) / 6.283185307179586476925286766559L;
      const long double part = turn - floorl(turn);  // in [0, 1)
      last.t.turns[k] = (uint64_t)(part * 18446744073709551616.0L);
    }
    last.base = base;
    last.d_R = d_R;
  }
  memcpy(t->turns, last.t.turns, (size_t)(d_R / 2) * sizeof(uint64_t));
}

// The append's tensor-core kernel: the widths its tiles are laid out for, groups
// that fit beside half a tile, and enough tokens that its start (W_c into TMEM,
// metadata) costs less than the generic kernel's arithmetic.  Generic against
// tensor cores, us: one sequence of 384 tokens 8.6 / 10.2, of 512 13.8 / 10.1, of
// 1024 20.7 / 10.5; one token of 256 sequences 10.2 / 15.0, of 512 18.2 / 15.4, of
// 1024 26.8 / 15.7.
constexpr int APPEND_TC_TOKENS = 512;
bool append_tc(const mtla_dims* d, int32_t N) {
  return d->dtype == MTLA_BF16 && d->r == 256 && d->d_R == 32 && d->s <= PTA_MAX_S && N >= APPEND_TC_TOKENS;
}

}  // namespace

extern "C" {

size_t mtla_paged_workspace_bytes(const mtla_dims* dims, int32_t B, int32_t N, int32_t which) {
  if (check_call_dims(dims) != MTLA_OK || B < 1 || N < 1 || which != MTLA_PAGED_ATTN) return 0;
  const AttnShape sh = attn_shape(dims);
  return sh.grid > 0 ? paged_layout(sh.grid, sh.rows, dims->r).total : 0;
}

mtla_status mtla_paged_append(const mtla_dims* dims, int32_t B, const mtla_chunk* chunk, const mtla_merge_args* merge,
                              double rope_base, const void* q_rope, void* q_rope_out, const mtla_paged_cache* cache,
                              const float* tail_in, float* tail_out, int32_t* t_out, int32_t* cache_len,
                              void* row_state, void* workspace, size_t workspace_bytes, int32_t* dev_err,
                              void* stream) {
  (void)workspace;
  (void)workspace_bytes;
  mtla_status st = check_call_dims(dims);
  if (st != MTLA_OK) return st;
  PagedAppendArgs a;
  if ((st = chunk_args(B, chunk, &a.c)) != MTLA_OK || (st = cache_args(dims, cache, &a.p)) != MTLA_OK) return st;
  if (!merge || !merge->W_c || !merge->b_c || !merge->P || merge->J_max < 1) return MTLA_ERR_INVALID_ARG;
  // (arrays without rows or columns may be null)
  if (chunk->N > 0 && (!merge->c_new || (!merge->kR_new && dims->d_R > 0))) return MTLA_ERR_INVALID_ARG;
  const void* ptrs[] = {merge->c_new, merge->kR_new, merge->W_c, merge->b_c, merge->P, row_state, q_rope, q_rope_out};
  for (const void* p : ptrs)
    if (!aligned(p, 16)) return MTLA_ERR_INVALID_ARG;
  if (!tail_in || !tail_out || !t_out || !dev_err || !aligned(tail_in, 4) || !aligned(tail_out, 4) ||
      !aligned(t_out, 4) || !aligned(cache_len, 4) || !aligned(dev_err, 4))
    return MTLA_ERR_INVALID_ARG;
  if (chunk->N > 0 && dims->d_R > 0 && (q_rope == nullptr) != (q_rope_out == nullptr)) return MTLA_ERR_INVALID_ARG;
  if (!(rope_base == 0.0 || (rope_base > 0.0 && isfinite(rope_base)))) return MTLA_ERR_INVALID_ARG;
  if (rope_base > 0.0 && dims->d_R % 2) return MTLA_ERR_UNSUPPORTED;
  const size_t D = dims->r + dims->d_R;
  if (overlap(tail_in, (size_t)B * D * 4, tail_out, (size_t)B * D * 4) ||
      overlap(chunk->t_prev, (size_t)B * 4, t_out, (size_t)B * 4) ||
      (cache_len && overlap(chunk->t_prev, (size_t)B * 4, cache_len, (size_t)B * 4)))
    return MTLA_ERR_INVALID_ARG;
  if ((int64_t)chunk->N * dims->H >= (int64_t(1) << 31)) return MTLA_ERR_UNSUPPORTED;
  // queries are rotated in place or into an array of their own
  const size_t q_bytes = (size_t)chunk->N * dims->H * dims->d_R * elem(dims->dtype);
  if (q_rope && q_rope_out && q_rope != q_rope_out && overlap(q_rope, q_bytes, q_rope_out, q_bytes)) return MTLA_ERR_INVALID_ARG;
  if (B == 0) return MTLA_OK;
  a.m.c_new = merge->c_new;
  a.m.kR_new = merge->kR_new;
  a.m.W_c = merge->W_c;
  a.m.b_c = merge->b_c;
  a.m.P = merge->P;
  a.m.J_max = merge->J_max;
  a.rotate = rope_base > 0.0 && dims->d_R > 0;
  if (a.rotate) rope_table(rope_base, dims->d_R, &a.rope);
  a.q_rope = chunk->N > 0 && dims->d_R > 0 ? q_rope : nullptr;
  a.q_rope_out = q_rope_out;
  a.tail_in = tail_in;
  a.tail_out = tail_out;
  a.t_out = t_out;
  a.cache_len = cache_len;
  a.row_state = row_state;
  a.dev_err = dev_err;
  a.H = dims->H;
  a.r = dims->r;
  a.d_R = dims->d_R;
  a.s = dims->s;
  a.div_s = fast_div((uint32_t)dims->s);
  const int sms = current_device_sms();
  if (sms <= 0) return MTLA_ERR_CUDA;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  if (append_tc(dims, chunk->N)) {
    PagedAppendMaps maps;
    const cuuint64_t dc[2] = {256, (cuuint64_t)chunk->N}, sc[1] = {512}, dk[2] = {32, (cuuint64_t)chunk->N}, sk[1] = {64};
    const cuuint32_t bc[2] = {64, 128}, bk[2] = {32, 128};
    if (!encode_bf16_tiled_map(&maps.c, merge->c_new, 2, dc, sc, bc, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode_bf16_tiled_map(&maps.kr, merge->kR_new, 2, dk, sk, bk, CU_TENSOR_MAP_SWIZZLE_NONE))
      return MTLA_ERR_CUDA;
    return from_cuda(launch_paged_append_tc(a, maps, sms, cs));
  }
  return from_cuda(launch_paged_append_simt(a, dims->dtype, sms, cs));
}

mtla_status mtla_paged_attn(const mtla_dims* dims, int32_t B, const mtla_chunk* chunk, const void* q_abs,
                            const void* q_rope, const void* row_state, const mtla_paged_cache* cache, void* out,
                            int32_t out_dtype, float* lse, void* workspace, size_t workspace_bytes, int32_t* dev_err,
                            void* stream) {
  mtla_status st = check_call_dims(dims);
  if (st != MTLA_OK) return st;
  PagedAttnArgs a;
  if ((st = chunk_args(B, chunk, &a.c)) != MTLA_OK || (st = cache_args(dims, cache, &a.p)) != MTLA_OK) return st;
  if (!dev_err) return MTLA_ERR_INVALID_ARG;
  if (chunk->N > 0 && (!q_abs || (!q_rope && dims->d_R > 0) || !row_state || !out)) return MTLA_ERR_INVALID_ARG;
  const void* ptrs[] = {q_abs, q_rope, row_state, out};
  for (const void* p : ptrs)
    if (!aligned(p, 16)) return MTLA_ERR_INVALID_ARG;
  if (!aligned(lse, 4) || !aligned(dev_err, 4)) return MTLA_ERR_INVALID_ARG;
  if (out_dtype != dims->dtype && out_dtype != MTLA_F32) return MTLA_ERR_INVALID_ARG;
  if ((int64_t)chunk->N * dims->H >= (int64_t(1) << 31)) return MTLA_ERR_UNSUPPORTED;
  if (B == 0 || chunk->N == 0) return MTLA_OK;
  const AttnShape sh = attn_shape(dims);
  if (sh.grid <= 0) return MTLA_ERR_CUDA;
  const PagedLayout l = paged_layout(sh.grid, sh.rows, dims->r);
  if (!workspace || !aligned(workspace, 16) || workspace_bytes < l.total) return MTLA_ERR_WORKSPACE;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  a.part.desc = reinterpret_cast<SplitDesc*>(ws + l.desc);
  a.part.ml = reinterpret_cast<float2*>(ws + l.ml);
  a.part.o = reinterpret_cast<float*>(ws + l.o);
  a.q_abs = q_abs;
  a.q_rope = q_rope;
  a.row_state = row_state;
  a.out = out;
  a.lse = lse;
  a.dev_err = dev_err;
  a.H = dims->H;
  a.r = dims->r;
  a.d_R = dims->d_R;
  a.out_f32 = out_dtype == MTLA_F32;
  a.rows = sh.rows;
  a.scale_log2 = (float)(1.4426950408889634 / sqrt((double)dims->d_h));
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  const int tpt = sh.rows / dims->H;
  a.plan.s = dims->s;
  a.plan.tpt = tpt < 16 ? tpt : 16;
  a.plan.q = (sh.tc ? PTC_COLS : PSN) / 8;
  // An item costs about three key tiles to start and to store; a share of its own
  // pays from about that weight on, and joining from somewhat more (tensor cores:
  // 14 sequences of one tile 10.0 us with shares of 3, 11.8 with 4, 10.0 with 2;
  // 1694 tokens of short sequences 29.6 with a cost of 3, 33.5 with 2; one sequence
  // of six tiles joined 12.1, in one block 13.0.  Generic kernel: two sequences of
  // 17 tokens 12.7 with shares of 1, 16.8 with 2; one token of one tile 8.7 alone
  // and 9.8 joined, of two 12.1 and 10.7).
  a.plan.item_cost = 3;
  a.plan.min_share = sh.tc ? 3 : 1;
  a.plan.one_block = sh.tc ? 8 : 4;
  a.plan.div_s = fast_div((uint32_t)dims->s);
  const int64_t rows = (int64_t)cache->table_pages * cache->page_rows;
  const int grid = most_blocks(a.plan, chunk->N, B, rows, sh.grid);
  if (sh.tc) {
    PagedAttnMaps maps;
    if (!paged_maps(&maps, a)) return MTLA_ERR_CUDA;
    if (launch_paged_attn_tc(a, maps, grid, cs) != cudaSuccess) return MTLA_ERR_CUDA;
  } else if (launch_paged_attn_simt(a, grid, dims->dtype, cs) != cudaSuccess) {
    return MTLA_ERR_CUDA;
  }
  // nothing to join where one block takes all, or no item has two tiles
  if (grid == 1 || most_tiles(a.plan, chunk->N, rows) <= 1) return MTLA_OK;
  return from_cuda(launch_paged_combine(a, grid, current_device_sms(), dims->dtype, cs));
}

mtla_status mtla_verify_drafts(int32_t B, int32_t N, int32_t V, const float* p, int64_t ld_p, const float* q,
                               int64_t ld_q, const int32_t* tokens, const int32_t* tok_start, const float* u_accept,
                               const float* u_sample, int32_t* n_keep, int32_t* next_token, int32_t* dev_err,
                               void* stream) {
  if (B < 0 || N < 0 || V < 1 || V > (1 << 22) || ld_p < V || (q && ld_q < V)) return MTLA_ERR_INVALID_ARG;
  if (!tok_start || !u_sample || !n_keep || !next_token || !dev_err) return MTLA_ERR_INVALID_ARG;
  if (N > 0 && (!p || !tokens || !u_accept)) return MTLA_ERR_INVALID_ARG;
  const void* ptrs[] = {p, q, tokens, tok_start, u_accept, u_sample, n_keep, next_token, dev_err};
  for (const void* x : ptrs)
    if (!aligned(x, 4)) return MTLA_ERR_INVALID_ARG;
  if (B == 0) return MTLA_OK;
  if (B >= (1 << 27)) return MTLA_ERR_UNSUPPORTED;
  VerifyArgs a;
  a.B = B;
  a.N = N;
  a.V = V;
  a.p = p;
  a.q = q;
  a.ld_p = ld_p;
  a.ld_q = ld_q;
  a.tokens = tokens;
  a.tok_start = tok_start;
  a.u_accept = u_accept;
  a.u_sample = u_sample;
  a.n_keep = n_keep;
  a.next_token = next_token;
  a.dev_err = dev_err;
  const int sms = current_device_sms();
  if (sms <= 0) return MTLA_ERR_CUDA;
  return from_cuda(launch_verify(a, sms, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
