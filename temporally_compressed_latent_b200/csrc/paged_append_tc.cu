// Appending a chunk of new tokens to a paged cache on the 5th-generation tensor
// cores (tcgen05 + TMEM): bf16, r = 256, d_R = 32, s <= 64, many tokens.
//
// What it computes: paged_append.cu's sums (MTLA paper notes, "Key designs:
// hyper-network temporal merging"),
//   S_t = [t opens its group ? 0 : S_{t-1}] + sigmoid((c W_c + b_c) * P[j-1]) * [c ; k^R].
//
// Design (B200):
//  * Transposed contraction D[channel, token] = W_c^T c^T: channels on the TMEM
//    lanes, so an epilogue thread owns one channel and the group sums run along
//    its own columns whatever sequences the tokens belong to.  The 288 channels
//    are three tiles of 96, one per CTA (MMA rows 96..127 are padding).
//  * W_c stays as exact as fp32 sums need: it is split into two bf16 parts
//    (W = hi + lo up to 2^-17 of it), both kept in TMEM as A operands, two MMAs
//    a K step.  The latents are bf16 already.  The tensor pipe has the room
//    (the epilogue's instructions bound the kernel), and the tail, which
//    travels between calls in fp32, keeps its 1e-6.
//  * A token tile is 128 consecutive token rows of which the first s - 1 repeat
//    the previous tile's last ones: a group that began there is summed again
//    from its start, so no CTA waits for another, and sums run in token order
//    from the group's start everywhere.
//  * A metadata warp works one tile ahead: it finds the tokens' sequences and
//    leaves, per token, its P row, its pool row (if it closes a group or its
//    chunk), its position and flags in shared memory.  The epilogue loads P and
//    the open groups' tails one chunk of 16 tokens ahead of their use.
//  * RoPE: an exact angle (double) every 8 tokens of a sequence and a rotation
//    by the pair's own angle between them (at most 7 single-precision
//    products: error below 2^-20 of the key).  The queries are rotated by the
//    epilogue warps while W_c and the first tiles are on their way.
#include "paged.cuh"

namespace mtla {
namespace ptp {

constexpr int R = 256, DR = 32, D = R + DR;
constexpr int CT = 3, NCT = D / CT;            // channel tiles of 96
constexpr int M = 128, NTOK = 128;             // MMA rows; token slots of a tile
constexpr int KB = R / 64;                     // K blocks of 64 latents
constexpr int BBLK = NTOK * 128;               // one K block of a tile: 16384 B
constexpr int KS = 2 * KB;                     // stages: two tiles
constexpr int KRBLK = NTOK * DR * 2;           // RoPE keys of a tile: 8192 B
constexpr int NWARPS = 16, NT = 32 * NWARPS;
constexpr int NEPI = 12;                       // epilogue warps: four per live lane quarter
constexpr int TMA_WARP = 3, MMA_WARP = 7, META_WARP = 11, SEQ_WARP = 15;  // warps of the padding quarter
constexpr uint32_t TMEM_COLS = 512, ACC_STRIDE = 128, HI_COL = 256, LO_COL = 384;
constexpr uint32_t IDESC = umma_idesc_bf16(M, NTOK, false, false);

// flags of a token
constexpr int F_TAKEN = 1;   // a sequence takes it
constexpr int F_OPEN = 2;    // the sum starts here (at tail_in with F_CARRY)
constexpr int F_CARRY = 4;
constexpr int F_LAST = 8;    // last token of its chunk
constexpr int F_BACK = 8;    // shift of: tokens of its group in the chunk before it

struct Meta {
  int4 tok[NTOK];   // P row, pool row or -1, position, flags
  int seq[NTOK];
};

constexpr size_t OFF_B = 0;
constexpr size_t OFF_KR = OFF_B + (size_t)KS * BBLK;
constexpr size_t OFF_META = OFF_KR + 2 * (size_t)KRBLK;
constexpr size_t OFF_ROPE = OFF_META + 2 * sizeof(Meta);
constexpr size_t OFF_BAR = OFF_ROPE + (DR / 2) * 8;
constexpr int NBAR = 2 * KS + 2 * 4 + 1;
constexpr size_t OFF_TMEM = OFF_BAR + NBAR * 8;
constexpr size_t SMEM = OFF_TMEM + 16 + 1024;
static_assert(SMEM <= 232448, "one block's shared memory (227 KB)");
static_assert(sizeof(Meta) % 16 == 0 && OFF_META % 16 == 0 && OFF_BAR % 8 == 0, "alignment");

__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity));
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr) : "memory");
}
__device__ __forceinline__ uint32_t tmem_ld1(uint32_t taddr) {
  uint32_t r;
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(r) : "r"(taddr) : "memory");
  return r;
}
// v sigmoid(z) = v / (1 + 2^y), y = -z log2 e (hardware base-2 exponential and
// reciprocal: relative error near 2^-22 each)
__device__ __forceinline__ float gated(float v, float y) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(y));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
  return v * r;
}
constexpr float kNegLog2e = -1.4426950408889634f;

// The sequences of token rows base + lane + 32 m, m < NM (b[m] = -1: none).
// A search for the first row, then the following starts 32 at a time.
template <int NM>
__device__ __forceinline__ void warp_sequences(const ChunkDev& c, int64_t base, int (&b)[NM]) {
  const int lane = threadIdx.x & 31;
  const int64_t first = base > 0 ? base : 0, last = base + 32 * NM - 1;
  int b0 = warp_find_seq(c.tok_start, c.B, (int)(first < c.N ? first : c.N));
#pragma unroll
  for (int m = 0; m < NM; ++m) b[m] = b0;
  for (int bb = b0 + 1; bb < c.B; bb += 32) {
    const int v = bb + lane < c.B ? c.tok_start[bb + lane] : 0x7fffffff;
    if (__shfl_sync(0xffffffffu, v, 0) > last) break;
    for (int k = 0; k < 32; ++k) {
      const int sk = __shfl_sync(0xffffffffu, v, k);
      if (sk > last) break;
#pragma unroll
      for (int m = 0; m < NM; ++m)
        if (sk <= base + lane + 32 * m) b[m] = bb + k;
    }
  }
}

// Rotate the queries of 32 token rows (or fewer) by one warp: lane l first finds
// row base + l's position; then two tokens a round, the 16 angles of each by
// one half of the warp, 16 bytes of a token a lane and step.
__device__ void rotate_queries(const PagedAppendArgs& a, int64_t base, int rows, const double* turns) {
  const int lane = threadIdx.x & 31;
  int b[1];
  warp_sequences<1>(a.c, base, b);
  int64_t pos = -1;
  if (lane < rows && base + lane < a.c.N && b[0] >= 0) {
    const AppendWin w = append_win(a, b[0], false);
    const int64_t place = base + lane - w.first;
    if (place < w.n) pos = w.t0 + place;
  }
  const int words = a.H * (DR / 8);  // 16-byte pieces of a token
  const uint4* src = reinterpret_cast<const uint4*>(a.q_rope);
  uint4* dst = reinterpret_cast<uint4*>(a.q_rope_out);
  for (int k = 0; k < rows; k += 2) {
    const int64_t p0 = __shfl_sync(0xffffffffu, pos, k), p1 = __shfl_sync(0xffffffffu, pos, k + 1 < 32 ? k + 1 : 31);
    const int64_t p[2] = {p0, k + 1 < rows ? p1 : -1};
    if (p[0] < 0 && p[1] < 0) continue;
    const int64_t mine = lane < 16 ? p[0] : p[1];
    const float2 cs = a.rotate ? rope_cos_sin(mine < 0 ? 0 : mine, turns[lane & 15]) : make_float2(1.f, 0.f);
    for (int w0 = 0; w0 < words; w0 += 32) {
      const int word = w0 + lane;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int64_t at = (base + k + h) * words + word;
        const bool on = p[h] >= 0 && word < words;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (on) v = src[at];
        uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {  // pair 4 (word mod 4) + e
          const int sl = 16 * h + 4 * (word & 3) + e;
          const float co = __shfl_sync(0xffffffffu, cs.x, sl), si = __shfl_sync(0xffffffffu, cs.y, sl);
          const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&x[e]));
          x[e] = pack_bf16x2(f.x * co - f.y * si, f.x * si + f.y * co);
        }
        if (on) dst[at] = make_uint4(x[0], x[1], x[2], x[3]);
      }
    }
  }
}

__global__ void __launch_bounds__(NT, 1) paged_append_tc_kernel(const __grid_constant__ PagedAppendMaps mp,
                                                                const __grid_constant__ PagedAppendArgs a, int n_tiles) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bar = reinterpret_cast<uint64_t*>(sm + OFF_BAR);
  uint64_t* const k_full = bar;                  // [KS]
  uint64_t* const k_empty = bar + KS;            // [KS]
  uint64_t* const acc_full = bar + 2 * KS;       // [2]
  uint64_t* const acc_empty = acc_full + 2;      // [2]
  uint64_t* const meta_full = acc_full + 4;      // [2]
  uint64_t* const meta_empty = acc_full + 6;     // [2]
  uint64_t* const mma_done = acc_full + 8;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(sm + OFF_TMEM);
  Meta* meta = reinterpret_cast<Meta*>(sm + OFF_META);
  double* turns = reinterpret_cast<double*>(sm + OFF_ROPE);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int ct = blockIdx.x % CT, G = gridDim.x / CT, j0 = blockIdx.x / CT;
  const int u_beg = (int)((int64_t)j0 * n_tiles / G), u_end = (int)((int64_t)(j0 + 1) * n_tiles / G);
  const bool has_rope = (ct + 1) * NCT > R;
  const int s = a.s, halo = s - 1, nout = NTOK - halo;
  const int q = warp & 3, part = warp >> 2;      // TMEM lane quarter; quarter of the tile's tokens
  const bool epi = q < 3;
  const int ch = ct * NCT + q * 32 + lane;       // this thread's channel (epilogue warps)

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // W_c^T: all of its loads in flight before anything else
  float wv[64];
  if (epi) {
#pragma unroll
    for (int k = 0; k < 64; ++k) wv[k] = __ldg(a.m.W_c + (size_t)(64 * part + k) * D + ch);
  }
  if (tid == 0) {
    for (int i = 0; i < KS; ++i) {
      mbar_init(&k_full[i], 1);
      mbar_init(&k_empty[i], NEPI);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], NEPI);
      mbar_init(&meta_full[i], 1);
      mbar_init(&meta_empty[i], NEPI);
    }
    mbar_init(mma_done, 1);
    fence_mbar_init();
  }
  if (tid < DR / 2) turns[tid] = a.rotate ? a.rope.turns[tid] : 0.0;
  if (warp == 0) {
    tmem_alloc(tmem_holder, TMEM_COLS);
    tmem_relinquish();
  }
  if (warp == TMA_WARP && lane == 0) {
    prefetch_tmap(&mp.c);
    prefetch_tmap(&mp.kr);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  bool ok = true;

  if (warp == TMA_WARP) {
    // ======================= TMA producer =======================
    if (lane == 0) {
      uint32_t kc = 0;
      for (int u = u_beg; u < u_end && ok; ++u) {
        const int32_t row = u * nout - halo;     // (rows before the first and past the last are zeros)
        const int b2 = ((u - u_beg) & 1);
        for (int kb = 0; kb < KB; ++kb, ++kc) {
          const int st = kc % KS;
          if (kc >= (uint32_t)KS && !mbar_wait(&k_empty[st], ((kc / KS) & 1) ^ 1)) { ok = false; break; }
          const bool kr = has_rope && kb == 0;   // the tile's RoPE keys ride with its first block
          mbar_arrive_expect_tx(&k_full[st], BBLK + (kr ? KRBLK : 0));
          tma_load_2d(sm + OFF_B + st * BBLK, &mp.c, kb * 64, row, &k_full[st]);
          if (kr) tma_load_2d(sm + OFF_KR + b2 * KRBLK, &mp.kr, 0, row, &k_full[st]);
        }
      }
      if (!ok) set_err(a.dev_err, MTLA_DEVERR_TIMEOUT);
      for (uint32_t i = kc > (uint32_t)KS ? kc - KS : 0; i < kc; ++i) mbar_wait(&k_full[i % KS], (i / KS) & 1);
    }
  } else if (warp == MMA_WARP) {
    // ======================= MMA issuer =======================
    named_bar(1, 32 * (NEPI + 1));               // W^T is in TMEM
    tc_fence_after();
    const uint32_t sB = smem_u32(sm + OFF_B);
    uint32_t kc = 0, tc = 0;
    for (int u = u_beg; u < u_end && ok; ++u, ++tc) {
      const int ab = tc & 1;
      if (tc >= 2 && !warp_wait(&acc_empty[ab], ((tc >> 1) & 1) ^ 1)) { ok = false; break; }
      tc_fence_after();
      const uint32_t dcol = tmem + ab * ACC_STRIDE;
      for (int kb = 0; kb < KB; ++kb, ++kc) {
        const int st = kc % KS;
        if (!warp_wait(&k_full[st], (kc / KS) & 1)) { ok = false; break; }
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            const uint64_t bd = umma_desc(sB + st * BBLK + kk * 32, 16, 1024, 2);
            umma_bf16_ts(dcol, tmem + HI_COL + (kb * 4 + kk) * 8, bd, IDESC, (kb > 0 || kk > 0) ? 1u : 0u);
            umma_bf16_ts(dcol, tmem + LO_COL + (kb * 4 + kk) * 8, bd, IDESC, 1u);
          }
        }
        __syncwarp();
      }
      if (!ok) break;
      if (elect_one()) umma_commit(&acc_full[ab]);
      __syncwarp();
    }
    if (!ok && lane == 0) set_err(a.dev_err, MTLA_DEVERR_TIMEOUT);
    if (elect_one()) umma_commit(mma_done);
    __syncwarp();
    warp_wait(mma_done, 0);
  } else if (warp == META_WARP) {
    // ======================= token metadata, one tile ahead =======================
    uint32_t tc = 0;
    for (int u = u_beg; u < u_end; ++u, ++tc) {
      const int mb = tc & 1;
      const int64_t base = (int64_t)u * nout - halo;
      int b[4];
      warp_sequences<4>(a.c, base, b);
      int4 t[4];
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const int64_t i = base + lane + 32 * m;
        t[m] = make_int4(0, -1, 0, 0);
        if (b[m] >= 0 && i >= 0 && i < a.c.N) {
          const AppendWin w = append_win(a, b[m], false);
          const int64_t place = i - w.first;
          if (place >= 0 && place < w.n) {
            const int64_t tm = w.t0 + place;     // 0-based time
            const int in = (int)(tm % s);
            const int64_t g = tm / s;
            t[m].x = (int)g;
            t[m].z = (int)tm;
            const bool last = place + 1 == w.n;
            t[m].w = F_TAKEN | (in == 0 || place == 0 ? F_OPEN : 0) | (in != 0 && place == 0 ? F_CARRY : 0) |
                     (last ? F_LAST : 0) | ((int)(in < place ? in : place) << F_BACK);
            if ((last || in + 1 == s) && lane + 32 * m >= halo) {
              t[m].y = (int)pool_row(a.p, b[m], g);
              if (t[m].y < 0) set_err(a.dev_err, MTLA_DEVERR_CAPACITY);
            }
          }
        }
      }
      if (tc >= 2 && !warp_wait(&meta_empty[mb], ((tc >> 1) & 1) ^ 1)) { ok = false; break; }
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        meta[mb].tok[lane + 32 * m] = t[m];
        meta[mb].seq[lane + 32 * m] = b[m];
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&meta_full[mb]);
    }
    if (!ok && lane == 0) set_err(a.dev_err, MTLA_DEVERR_TIMEOUT);
  } else if (warp == SEQ_WARP) {
    // ======================= per-sequence results =======================
    for (int b = blockIdx.x; b < a.c.B; b += gridDim.x) {
      const AppendWin w = append_win(a, b, lane == 0);
      if (lane == 0) {
        a.t_out[b] = (int32_t)(w.t0 + w.n);
        if (a.cache_len) a.cache_len[b] = w.t0 + w.n > 0 ? (int32_t)group_of(w.t0 + w.n, s) : 0;
      }
      if (w.n == 0)
        for (int k = lane; k < D; k += 32) a.tail_out[(int64_t)b * D + k] = a.tail_in[(int64_t)b * D + k];
    }
  } else {
    // ======================= epilogue warps =======================
    const bool rope = ch >= R;                   // warp-uniform
    const uint32_t lane_base = tmem + ((uint32_t)(q * 32) << 16);
    {
      // W^T as two bf16 parts into TMEM (loads issued at the kernel's start)
      uint32_t hi[32], lo[32];
#pragma unroll
      for (int k = 0; k < 32; ++k) {
        const float w0 = wv[2 * k], w1 = wv[2 * k + 1];
        hi[k] = pack_bf16x2(w0, w1);
        const float2 h = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&hi[k]));
        lo[k] = pack_bf16x2(w0 - h.x, w1 - h.y);
      }
      tmem_st32(lane_base + HI_COL + 32 * part, hi);
      tmem_st32(lane_base + LO_COL + 32 * part, lo);
      tmem_wait_st();
      tc_fence_before();
    }
    named_bar(1, 32 * (NEPI + 1));
    const float bc = __ldg(a.m.b_c + ch);
    const float* Pc = a.m.P + ch;
    const uint32_t sB = smem_u32(sm + OFF_B);
    // this channel's byte inside a swizzled 128-byte latent row (K block ch / 64)
    const uint32_t c_kb = (uint32_t)((ch & 255) >> 6), c_chunk = (uint32_t)((ch & 63) >> 3), c_in = (uint32_t)(ch & 7) * 2;
    const int pair = (ch & 31) >> 1;
    const double turn = rope ? turns[pair] : 0.0;
    const float2 step = rope ? rope_cos_sin(1, turn) : make_float2(1.f, 0.f);
    const float sgn = (ch & 1) ? 1.f : -1.f;     // odd channels: x1 cos + x0 sin; even: x0 cos - x1 sin
    __nv_bfloat16* const state = reinterpret_cast<__nv_bfloat16*>(a.row_state) + (a.row_state ? ch : 0);
    __nv_bfloat16* const pages = reinterpret_cast<__nv_bfloat16*>(a.p.pages) + ch;
    uint32_t tc = 0;
    bool queries = a.q_rope != nullptr;
    for (int u = u_beg; u < u_end || queries; ++u, ++tc) {
      if (queries) {
        // this warp's share of the queries, at most 32 rows at a time: before
        // the first tile, whose operands are still on their way
        queries = false;
        const int64_t warps = (int64_t)gridDim.x * NEPI;
        int64_t rows = (a.c.N + warps - 1) / warps;
        rows = rows < 32 ? (rows + 1) / 2 * 2 : 32;
        for (int64_t k = ((int64_t)blockIdx.x * NEPI + part * 3 + q) * rows; k < a.c.N; k += warps * rows)
          rotate_queries(a, k, (int)rows, turns);
        if (u >= u_end) break;
      }
      const int ab = tc & 1, sb = ab * KB;
      const uint32_t par = (tc >> 1) & 1;
      const int64_t base = (int64_t)u * nout - halo;
      if (!warp_wait(&meta_full[ab], par)) { ok = false; break; }
      const Meta& mt = meta[ab];
      const int cb = 32 * part > halo ? 32 * part : halo, ce = 32 * part + 32;
      const int64_t lastc = a.c.N - base;        // columns past it are no token rows
      const int hi_c = ce < lastc ? ce : (int)lastc;
      const int back = cb < hi_c ? mt.tok[cb].w >> F_BACK : 0;
      float run = 0.f;
      float2 cs = make_float2(1.f, 0.f);
      int cs_pos = -2, cs_seq = -1, cs_age = 0;  // position and sequence that cs holds
      // chunk loads: P and, where a sequence goes on in an open group, its tail
      float pn[16], tn[16];
      auto fetch = [&](int c0) {
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          const int4 t = mt.tok[c0 + k];
          pn[k] = __ldg(Pc + (int64_t)t.x * D);
          tn[k] = 0.f;
          if (t.w & F_CARRY) tn[k] = a.tail_in[(int64_t)mt.seq[c0 + k] * D + ch];
        }
      };
      // the key entry of a column: the rotated pair, fp32
      auto key = [&](int col, const int4& t) -> float {
        const uint32_t row = smem_u32(sm + OFF_KR + ab * KRBLK) + (uint32_t)col * (DR * 2) + (uint32_t)(ch & 31) * 2;
        uint16_t own, other;
        asm volatile("ld.shared.u16 %0, [%1];" : "=h"(own) : "r"(row));
        if (!a.rotate) return __bfloat162float(__ushort_as_bfloat16(own));
        asm volatile("ld.shared.u16 %0, [%1];" : "=h"(other) : "r"(row ^ 2u));
        const int sq = mt.seq[col];
        if (sq != cs_seq || t.z != cs_pos + 1 || cs_age == 7) {
          cs = rope_cos_sin(t.z, turn);
          cs_age = 0;
        } else {
          cs = make_float2(cs.x * step.x - cs.y * step.y, cs.x * step.y + cs.y * step.x);
          ++cs_age;
        }
        cs_pos = t.z;
        cs_seq = sq;
        return __bfloat162float(__ushort_as_bfloat16(own)) * cs.x + sgn * __bfloat162float(__ushort_as_bfloat16(other)) * cs.y;
      };
      auto latent = [&](int col) -> float {
        uint16_t raw;
        const uint32_t at = sB + (sb + c_kb) * BBLK + (uint32_t)(col >> 3) * 1024 + (uint32_t)(col & 7) * 128 +
                            ((c_chunk ^ (uint32_t)(col & 7)) << 4) + c_in;
        asm volatile("ld.shared.u16 %0, [%1];" : "=h"(raw) : "r"(at));
        return __bfloat162float(__ushort_as_bfloat16(raw));
      };
      if (cb < hi_c) fetch(cb & ~15);
      ok = warp_wait(&acc_full[ab], par) && warp_wait(&k_full[sb], par) && warp_wait(&k_full[sb + c_kb], par);
      tc_fence_after();
      if (!ok) break;
      // the first group's earlier tokens, summed again from its start
      for (int col = cb - back; col < cb && cb < hi_c; ++col) {
        const int4 t = mt.tok[col];
        const float g = __uint_as_float(tmem_ld1(lane_base + ab * ACC_STRIDE + col));
        const float pa = __ldg(Pc + (int64_t)t.x * D) * kNegLog2e;
        const float x = rope ? key(col, t) : latent(col);
        float start = run;
        if (t.w & F_OPEN) start = t.w & F_CARRY ? a.tail_in[(int64_t)mt.seq[col] * D + ch] : 0.f;
        tmem_wait_ld();
        run = start + gated(x, fmaf(g, pa, bc * pa));
      }
      for (int c0 = cb & ~15; c0 < hi_c; c0 += 16) {
        uint32_t g[16];
        tmem_ld16(lane_base + ab * ACC_STRIDE + c0, g);
        float v[16], pc[16], tl[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          pc[k] = pn[k];
          tl[k] = tn[k];
        }
        if (c0 + 16 < hi_c) fetch(c0 + 16);
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          if (rope) {
            v[k] = 0.f;
            if (c0 + k >= cb && c0 + k < hi_c) v[k] = key(c0 + k, mt.tok[c0 + k]);
          } else {
            v[k] = latent(c0 + k);
          }
        }
        tmem_wait_ld();
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          const float pa = pc[k] * kNegLog2e;
          v[k] = gated(v[k], fmaf(__uint_as_float(g[k]), pa, bc * pa));
        }
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          const int col = c0 + k;
          if (col >= cb && col < hi_c) {
            const int4 t = mt.tok[col];
            run = (t.w & F_OPEN ? tl[k] : run) + v[k];
            if (t.w & F_TAKEN) {
              const __nv_bfloat16 o = __float2bfloat16_rn(run);
              if (a.row_state) state[(base + col) * D] = o;
              if (t.y >= 0) pages[(int64_t)t.y * a.p.row_stride] = o;
              if (t.w & F_LAST) a.tail_out[(int64_t)mt.seq[col] * D + ch] = run;
            }
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&acc_empty[ab]);
        mbar_arrive(&meta_empty[ab]);
        for (int kb = 0; kb < KB; ++kb) mbar_arrive(&k_empty[sb + kb]);
      }
    }
    if (!ok && lane == 0) set_err(a.dev_err, MTLA_DEVERR_TIMEOUT);
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, TMEM_COLS);
  }
}

}  // namespace ptp

cudaError_t launch_paged_append_tc(const PagedAppendArgs& a, const PagedAppendMaps& m, int sms, cudaStream_t st) {
  static uint64_t done_mask = 0;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !(done_mask & (1ull << dev))) {
    e = cudaFuncSetAttribute(ptp::paged_append_tc_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)ptp::SMEM);
    if (e != cudaSuccess) return e;
    if (dev < 64) done_mask |= 1ull << dev;
  }
  const int n_tiles = (int)cdiv(a.c.N, ptp::NTOK - (a.s - 1));
  int per = sms / ptp::CT > 0 ? sms / ptp::CT : 1;  // CTAs per channel tile
  if (n_tiles < per) per = n_tiles;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(ptp::CT * per));
  cfg.blockDim = dim3(ptp::NT);
  cfg.dynamicSmemBytes = ptp::SMEM;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, ptp::paged_append_tc_kernel, m, a, n_tiles);
}

}  // namespace mtla
