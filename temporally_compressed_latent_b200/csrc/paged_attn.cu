// Attention of a chunk of new tokens over a paged cache: the generic kernel
// (any supported H, r, d_R; fp32 or bf16 storage, fp32 arithmetic) and the
// kernel that combines the parts of split items (shared with the tensor-core
// kernel in paged_attn_tc.cu).
//
// What it computes (MTLA paper notes, "Key designs: stride-aware causal mask"
// and "decoupled RoPE with temporal compression"; Figure 2(c) of the abstract
// page): the query of a token at time t attends the complete groups before its
// own (cache rows 0 .. ceil(t/s) - 2) and its own state row; one pass over the
// columns with a running maximum and sum per row,
//   m' = max(m, x),  l' = l 2^(m - m') + sum 2^(x - m'),  O' = O 2^(m - m') + P C_hat,
// x in log2 units.  The own states are virtual key rows behind the cache rows,
// so every row that is stored has at least one visible column.
//
// A block walks its share of the items (paged.cuh): 32 (token, head) rows of a
// sequence against key tiles of 32 rows, which asynchronous copies bring two
// tiles ahead (table entries one more).  The scores take 2 x 2 per thread from
// shared memory with four-wide loads, the values 4 rows x 4 n channels per
// thread with the running output in registers, two products an instruction
// (packed fp32); rows of up to 64 latents leave half of a warp's lanes to take
// the tile's other keys.  Issue bounds it where a chunk is long, the chain of a
// tile's steps where it is short.
#include "paged.cuh"

namespace mtla {
namespace psimt {

constexpr int NT = 256;
constexpr int WINS = 64;  // windows kept (the widest rows leave no more room)

// key rows in shared memory: 4 elements more than the row, so that reads of 16
// rows touch every bank group once
__host__ __device__ constexpr int key_pitch(int D, int elem) { return (D + 16 / elem) * elem; }
constexpr size_t smem_bytes(int D, int elem) {
  return (size_t)PSM * (D + 4) * 4 + (size_t)2 * PSN * key_pitch(D, elem) + (size_t)PSN * (PSM + 4) * 4 + PSM * 4 * 3 +
         sizeof(PlanShared) + WINS * sizeof(SeqWin) + 32 * sizeof(ItemWalk) + sizeof(Item) + 64;
}
constexpr int MAXD = 576;  // r + d_R
static_assert(smem_bytes(MAXD, 4) <= 232448, "the widest fp32 rows have to fit a block");

template <typename T> __device__ __forceinline__ void ld4(const T* p, float* v);
template <> __device__ __forceinline__ void ld4<float>(const float* p, float* v) {
  const float4 x = *reinterpret_cast<const float4*>(p);
  v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
}
template <> __device__ __forceinline__ void ld4<__nv_bfloat16>(const __nv_bfloat16* p, float* v) {
  const uint2 x = *reinterpret_cast<const uint2*>(p);
  const float2 a = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&x.x));
  const float2 b = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&x.y));
  v[0] = a.x; v[1] = a.y; v[2] = b.x; v[3] = b.y;
}

template <typename T> __device__ __forceinline__ float4 ld4v(const T* p) {
  float v[4];
  ld4(p, v);
  return make_float4(v[0], v[1], v[2], v[3]);
}

// two fp32 products and sums in one instruction
__device__ __forceinline__ uint64_t pack2(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// Zeros in the place of a key tile's latents that are not finite, in its virtual
// rows from `from` on (those below are seen by every row of the item).  The
// block's barrier after the softmax comes before the value product.
template <typename T>
static __device__ __noinline__ void hide_latents(uint8_t* tile, int pitch, int r, uint32_t v0, uint32_t from) {
  const int words = r * (int)sizeof(T) / 4;
  for (int k = threadIdx.x >> 5; k < PSN; k += NT / 32) {
    if (v0 + k < from) continue;
    uint32_t* const row = reinterpret_cast<uint32_t*>(tile + k * pitch);
    for (int e = threadIdx.x & 31; e < words; e += 32) row[e] = finite_or_zero<T>(row[e]);
  }
}

// NQ: channel quads per lane, ceil(r / 128); 0: r <= 64, where lanes 16 .. 31
// take every second key.  Three blocks an SM where the running output is small
// (8 sequences of up to 33 tokens over 500 rows, r = 64: 19.1 us; two blocks
// 21.7, four, whose registers spill, 21.9).
template <typename T, int NQ0>
__global__ void __launch_bounds__(NT, NQ0 < 2 ? 3 : (NQ0 == 2 ? 2 : 1)) paged_attn_simt_kernel(const __grid_constant__ PagedAttnArgs a) {
  constexpr int NQ = NQ0 > 0 ? NQ0 : 1, NK = NQ0 > 0 ? 1 : 2;  // channel quads; key groups of a warp
  const int kg = NK == 2 ? (int)(threadIdx.x & 31) >> 4 : 0, cl = NK == 2 ? (int)threadIdx.x & 15 : (int)threadIdx.x & 31;
  extern __shared__ float smem[];
  const int D = a.r + a.d_R, DP = D + 4, KP = key_pitch(D, sizeof(T)), KT = KP / (int)sizeof(T);
  float* Qs = smem;                       // [PSM][DP]
  uint8_t* Kb = reinterpret_cast<uint8_t*>(Qs + PSM * DP);              // [2][PSN rows of KP bytes]
  float* Ss = reinterpret_cast<float*>(Kb + 2 * PSN * KP);              // [PSN][PSM + 4]: probabilities, key-major
  float* sm_m = Ss + PSN * (PSM + 4);     // [PSM] running maxima
  float* sm_l = sm_m + PSM;               // [PSM] running sums
  float* sm_a = sm_l + PSM;               // [PSM] rescale factors of the current tile
  PlanShared* plan = reinterpret_cast<PlanShared*>((reinterpret_cast<uintptr_t>(sm_a + PSM) + 15) & ~uintptr_t(15));
  SeqWin* wins = reinterpret_cast<SeqWin*>(plan + 1);
  ItemWalk* walks = reinterpret_cast<ItemWalk*>(wins + WINS);  // the first warp's, a lane each: no registers between items
  Item* sit = reinterpret_cast<Item*>(walks + 32);
  int* more = reinterpret_cast<int*>(sit + 1);
  int* hid = more + 1;                    // a score that its row does not see is not finite (see restore_nan)
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int grid = gridDim.x, x = blockIdx.x;

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  plan_block<NT, WINS>(a.c, a.p, a.plan, grid, x, a.dev_err, plan, wins);
  if (warp == 0) {
    walks[lane].init(a.c, a.p, a.plan, x, plan, wins);
    if (lane == 0) a.part.desc[x] = {0, 0, 0, 0};
  }

  for (;;) {
    if (warp == 0) {
      Item it;
      ItemWalk walk = walks[lane];
      const bool any = walk.next(a.c, a.p, a.plan, &it);
      walks[lane] = walk;
      if (lane == 0) {
        *more = any;
        *hid = 0;
        if (any) *sit = it;
      }
      if (any && it.slot >= 0 && it.kt1 == it.kt && lane == 0)  // a split item ends here
        a.part.desc[x] = {it.row0, it.ntok, first_block(a.plan, walk.C, walk.G, walk.item_start), 0};
    }
    __syncthreads();
    if (!*more) break;
    const Item& it = *sit;
    const int live = it.ntok * a.H;
    const uint32_t R = (uint32_t)it.R, R8 = (R + 7) & ~7u;  // (below 2^31)
    if (tid < PSM) {
      sm_m[tid] = -INFINITY;
      sm_l[tid] = 0.f;
    }
    uint64_t o[4][NQ * 2];                       // rows 4 warp + i, channel pairs
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int c = 0; c < NQ * 2; ++c) o[i][c] = 0;

    // keys: cache rows, then the tokens' own states; rows between and behind
    // them are zeros.  A warp brings rows warp, warp + 8, ... of a tile; lane l
    // of it looks up row (l mod 4)'s page a tile ahead.
    constexpr int RW = PSN / (NT / 32);           // rows a warp (4)
    const int chunks = D * (int)sizeof(T) / 16;   // 16-byte pieces of a row
    auto look = [&](int kt) -> int64_t {          // pool row, -1: zeros, or -2 - token: an own state
      const uint32_t g = (uint32_t)kt * PSN + warp + (lane % RW) * (NT / 32);
      if (g < R) {
        const int64_t row = pool_row(a.p, it.b, g);
        if (row < 0) set_err(a.dev_err, MTLA_DEVERR_CAPACITY);
        return row;
      }
      return g - R8 < (uint32_t)it.ntok ? -2 - (int64_t)it.row0 - (int64_t)(g - R8) : -1;
    };
    auto copy = [&](int64_t at, int buf) {
#pragma unroll
      for (int k = 0; k < RW; ++k) {
        const int64_t row = __shfl_sync(0xffffffffu, at, k);
        const T* src = row >= 0 ? reinterpret_cast<const T*>(a.p.pages) + row * a.p.row_stride
                                : reinterpret_cast<const T*>(a.row_state) + (row == -1 ? 0 : -2 - row) * D;
        const uint32_t dst = smem_u32(Kb + (buf * PSN + warp + k * (NT / 32)) * KP);
        const int bytes = row == -1 ? 0 : 16;     // (0: the piece is filled with zeros)
        for (int c = lane; c < chunks; c += 32)
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + c * 16),
                       "l"(reinterpret_cast<const uint8_t*>(src) + c * 16), "r"(bytes) : "memory");
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    // queries (rows past the live ones: zeros), eight threads a row; read while
    // the first tile's rows are looked up
    const int qi = tid >> 3;
    const bool q_live = qi < live;
    const int64_t q_row = (int64_t)it.row0 * a.H + qi;
    auto q_quad = [&](int e) {
      if (!q_live || e >= D) return make_float4(0.f, 0.f, 0.f, 0.f);
      return e < a.r ? ld4v(reinterpret_cast<const T*>(a.q_abs) + q_row * a.r + e)
                     : ld4v(reinterpret_cast<const T*>(a.q_rope) + q_row * a.d_R + (e - a.r));
    };
    float4 qv[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) qv[k] = q_quad(4 * (tid & 7) + 32 * k);
    copy(look(it.kt0), 0);
    for (int e0 = 4 * (tid & 7); e0 < D; e0 += 128) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (e0 + 32 * k < D) *reinterpret_cast<float4*>(Qs + qi * DP + e0 + 32 * k) = qv[k];
        if (e0 + 128 < D) qv[k] = q_quad(e0 + 128 + 32 * k);
      }
    }
    // scores: this thread's rows r0, r0 + 16 (token, cache rows below it, virtual
    // row of its own state; a row past the live ones sees nothing)
    const int r0 = tid >> 4, c0 = tid & 15;
    uint32_t seen[2], own[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int tok = (r0 + 16 * k) / a.H;
      seen[k] = tok < it.ntok ? rows_below(a.plan, it.t + tok) : 0;
      own[k] = tok < it.ntok ? R8 + tok : 0xffffffffu;
    }
    int64_t ahead = it.kt0 + 1 < it.kt1 ? look(it.kt0 + 1) : -1;

    for (int kt = it.kt0; kt < it.kt1; ++kt) {
      const uint32_t v0 = (uint32_t)kt * PSN;     // first virtual row
      const T* Ks = reinterpret_cast<const T*>(Kb + ((kt - it.kt0) & 1) * PSN * KP);
      if (kt + 1 < it.kt1) {
        copy(ahead, (kt + 1 - it.kt0) & 1);
        ahead = kt + 2 < it.kt1 ? look(kt + 2) : -1;
        asm volatile("cp.async.wait_group 1;" ::: "memory");
      } else {
        asm volatile("cp.async.wait_group 0;" ::: "memory");
      }
      __syncthreads();
      // scores: rows r0, r0 + 16; keys c0, c0 + 16
      uint64_t t00 = 0, t01 = 0, t10 = 0, t11 = 0;
#pragma unroll 2
      for (int e = 0; e < D; e += 4) {
        const ulonglong2 q0 = *reinterpret_cast<const ulonglong2*>(Qs + r0 * DP + e);
        const ulonglong2 q1 = *reinterpret_cast<const ulonglong2*>(Qs + (r0 + 16) * DP + e);
        const float4 f0 = ld4v(Ks + c0 * KT + e), f1 = ld4v(Ks + (c0 + 16) * KT + e);
        const uint64_t k0x = pack2(f0.x, f0.y), k0y = pack2(f0.z, f0.w), k1x = pack2(f1.x, f1.y), k1y = pack2(f1.z, f1.w);
        t00 = fma2(q0.y, k0y, fma2(q0.x, k0x, t00));
        t01 = fma2(q0.y, k1y, fma2(q0.x, k1x, t01));
        t10 = fma2(q1.y, k0y, fma2(q1.x, k0x, t10));
        t11 = fma2(q1.y, k1y, fma2(q1.x, k1x, t11));
      }
      auto both = [](uint64_t v) { const float2 f = unpack2(v); return f.x + f.y; };
      const float s00 = both(t00), s01 = both(t01), s10 = both(t10), s11 = both(t11);
      auto put = [&](int k, int c, float v) {
        const uint32_t g = v0 + c;
        const bool sees = g < seen[k] || g == own[k];
        Ss[c * (PSM + 4) + r0 + 16 * k] = sees ? v * a.scale_log2 : -INFINITY;
        if (!sees && own[k] != 0xffffffffu && !isfinite(v) && (g < R || g - R8 < (uint32_t)it.ntok)) *hid = 1;
      };
      put(0, c0, s00);
      put(0, c0 + 16, s01);
      put(1, c0, s10);
      put(1, c0 + 16, s11);
      __syncthreads();
      if (*hid) hide_latents<T>(Kb + ((kt - it.kt0) & 1) * PSN * KP, KP, a.r, v0, rows_below(a.plan, it.t));
      {  // softmax: eight lanes a row, four keys each
        const int i = tid >> 3, k0 = tid & 7;
        float xv[4], mx = -INFINITY;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          xv[k] = Ss[(k0 + 8 * k) * (PSM + 4) + i];
          mx = fmaxf(mx, xv[k]);
        }
#pragma unroll
        for (int d = 4; d > 0; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
        const float mo = sm_m[i], mn = fmaxf(mo, mx), ref = mn == -INFINITY ? 0.f : mn;
        float sum = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float p = exp2f(xv[k] - ref);  // exp2f(-inf) = 0
          Ss[(k0 + 8 * k) * (PSM + 4) + i] = p;
          sum += p;
        }
#pragma unroll
        for (int d = 4; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        __syncwarp();
        if (k0 == 0) {
          const float f = exp2f(mo - ref);     // 0 while nothing was visible
          sm_a[i] = f;
          sm_m[i] = mn;
          sm_l[i] = sm_l[i] * f + sum;
        }
      }
      __syncthreads();
      // values: this warp's rows 4 warp .. + 3, channels 4 cl + 128 q
      if (4 * warp < live) {
        const float4 f = *reinterpret_cast<const float4*>(sm_a + 4 * warp);
        const uint64_t fa[4] = {pack2(f.x, f.x), pack2(f.y, f.y), pack2(f.z, f.z), pack2(f.w, f.w)};
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int c = 0; c < NQ * 2; ++c) o[i][c] = mul2(o[i][c], fa[i]);
#pragma unroll 4
        for (int k = kg; k < PSN; k += NK) {
          const float4 p4 = *reinterpret_cast<const float4*>(Ss + k * (PSM + 4) + 4 * warp);
          const uint64_t pv[4] = {pack2(p4.x, p4.x), pack2(p4.y, p4.y), pack2(p4.z, p4.z), pack2(p4.w, p4.w)};
#pragma unroll
          for (int q = 0; q < NQ; ++q) {
            const int e = 4 * cl + 128 * q;
            if (e < a.r) {
              const float4 c4 = ld4v(Ks + k * KT + e);
              const uint64_t cx = pack2(c4.x, c4.y), cy = pack2(c4.z, c4.w);
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                o[i][2 * q] = fma2(pv[i], cx, o[i][2 * q]);
                o[i][2 * q + 1] = fma2(pv[i], cy, o[i][2 * q + 1]);
              }
            }
          }
        }
      }
      __syncthreads();
    }
    if (NK == 2) {  // the two key groups' sums
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int c = 0; c < NQ * 2; ++c) {
          const float2 v = unpack2(o[i][c]);
          o[i][c] = pack2(v.x + __shfl_xor_sync(0xffffffffu, v.x, 16), v.y + __shfl_xor_sync(0xffffffffu, v.y, 16));
        }
    }
    // the item's rows out: finished, or as a part
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = 4 * warp + i;
      if (row < live && kg == 0) {
        const float m = sm_m[row], l = sm_l[row];
        const int64_t orow = (int64_t)it.row0 * a.H + row, prow = (int64_t)it.slot * a.rows + row;
        const float inv = it.slot < 0 ? 1.f / l : 1.f;
        if (lane == 0) {
          if (it.slot >= 0) a.part.ml[prow] = make_float2(m, l);
          else if (a.lse) a.lse[orow] = (m + log2f(l)) * 0.6931471805599453f;
        }
#pragma unroll
        for (int q = 0; q < NQ; ++q) {
          const int e = 4 * cl + 128 * q;
          if (e < a.r) {
            const float2 x = unpack2(o[i][2 * q]), y = unpack2(o[i][2 * q + 1]);
            const float4 v = make_float4(x.x * inv, x.y * inv, y.x * inv, y.y * inv);
            if (it.slot >= 0) *reinterpret_cast<float4*>(a.part.o + prow * a.r + e) = v;
            else if (a.out_f32 || sizeof(T) == 4) *reinterpret_cast<float4*>(reinterpret_cast<float*>(a.out) + orow * a.r + e) = v;
            else
              *reinterpret_cast<uint2*>(reinterpret_cast<__nv_bfloat16*>(a.out) + orow * a.r + e) =
                  make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
          }
        }
      }
    }
    if (*hid && 4 * warp < live) {
      const bool f32 = it.slot >= 0 || a.out_f32 || sizeof(T) == 4;
      const int64_t first = it.slot >= 0 ? (int64_t)it.slot * a.rows : (int64_t)it.row0 * a.H;
      void* const dst = it.slot >= 0 ? (void*)(a.part.o + first * a.r)
                                     : (f32 ? (void*)(reinterpret_cast<float*>(a.out) + first * a.r)
                                            : (void*)(reinterpret_cast<T*>(a.out) + first * a.r));
      restore_nan<T>(a, it.b, it.row0, it.t, 4 * warp, live < 4 * warp + 4 ? live : 4 * warp + 4, dst, f32);
    }
    __syncthreads();  // the item and its statistics have been read
  }
}

// ----------------------------------------------------------------------------
// Combine: block (x, y) finishes rows of the split item that ends in block x of
// the attention grid, or of the x-th one (`nth`, see launch_paged_combine):
//   out = sum_x 2^(m_x - M) O_x / sum_x 2^(m_x - M) l_x
// over its parts x.  A row takes a warp, eight channels a lane and three parts
// in flight (the loads' latency bounds a decode step's few rows, the
// instructions a long chunk's many: with 64 threads a row the latter took half
// as long again), or two or four warps, which share its parts, where there are
// more parts than that and blocks enough for all rows at once.  At 64 registers a thread a block fits beside the attention's and waits there for its
// end.
// ----------------------------------------------------------------------------
constexpr int CNT = 128, CNW = CNT / 32, CNP = 3;

template <typename T>
__global__ void __launch_bounds__(CNT, 8) paged_combine_kernel(const __grid_constant__ PagedAttnArgs a, int nth) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  __shared__ float4 red[CNW][2][32];
  __shared__ float2 red_ml[CNW];
  __shared__ uint32_t ends[4 * CNW];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int g = blockIdx.x;
  if (nth > 0) {  // the x-th of the nth notes that is not empty
    int left = blockIdx.x;
    g = -1;
    for (int g0 = 0; g0 < nth && g < 0; g0 += 4 * CNT) {
      bool some[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int at = g0 + k * CNT + (int)threadIdx.x;
        some[k] = at < nth && a.part.desc[at].ntok > 0;
      }
      if (g0 > 0) __syncthreads();
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t m = __ballot_sync(0xffffffffu, some[k]);
        if (lane == 0) ends[k * CNW + warp] = m;
      }
      __syncthreads();
      for (int w = 0; w < 4 * CNW; ++w) {
        uint32_t m = ends[w];
        const int c = __popc(m);
        if (left < c) {
          for (; left > 0; --left) m &= m - 1;
          g = g0 + 32 * w + __ffs(m) - 1;
          break;
        }
        left -= c;
      }
    }
    if (g < 0) return;
  }
  const SplitDesc* const d = a.part.desc + g;
  const int live = d->ntok * a.H;
  if (live == 0) return;
  const int first = d->first, parts = g - first + 1;  // every block between has one (their shares are not empty)
  const int64_t row0 = (int64_t)d->row0 * a.H;
  int W = 1;  // warps a row
  while (W < CNW && W * CNP < parts && live * 2 * W <= CNW * (int)gridDim.y) W *= 2;
  const int sub = warp % W, rows_at_once = CNW / W;
  for (int r0 = blockIdx.y * rows_at_once; r0 < live; r0 += gridDim.y * rows_at_once) {
    const int row = r0 + warp / W;
    for (int e0 = 0; e0 < a.r; e0 += 256) {
      const int e = e0 + 4 * lane;  // and e + 128
      const bool on0 = row < live && e < a.r, on1 = row < live && e + 128 < a.r;
      float M = -INFINITY, L = 0.f;
      float4 acc[2] = {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
      for (int k0 = sub; row < live && k0 < parts; k0 += CNP * W) {
        float2 ml[CNP];
        float4 o[CNP][2];
        float Mn = M;
#pragma unroll
        for (int u = 0; u < CNP; ++u) {
          const int k = k0 + u * W;
          ml[u] = make_float2(-INFINITY, 0.f);
          o[u][0] = o[u][1] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (k < parts) {
            const int64_t prow = (int64_t)(2 * (first + k) + (k == 0 ? 1 : 0)) * a.rows + row;
            ml[u] = a.part.ml[prow];
            const float* const src = a.part.o + prow * a.r + e;
            if (on0) o[u][0] = *reinterpret_cast<const float4*>(src);
            if (on1) o[u][1] = *reinterpret_cast<const float4*>(src + 128);
          }
        }
#pragma unroll
        for (int u = 0; u < CNP; ++u) Mn = fmaxf(Mn, ml[u].x);
        const float ref = Mn == -INFINITY ? 0.f : Mn, f = exp2f(M - ref);
        M = Mn;
        L *= f;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          acc[h].x *= f; acc[h].y *= f; acc[h].z *= f; acc[h].w *= f;
        }
#pragma unroll
        for (int u = 0; u < CNP; ++u) {
          // (a part with nothing visible to this row has m = -inf and zeros; one
          // whose only visible scores are NaN has m = -inf too, and its NaN stays)
          const float w = exp2f(ml[u].x - ref);
          L = fmaf(ml[u].y, w, L);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            acc[h].x = fmaf(o[u][h].x, w, acc[h].x);
            acc[h].y = fmaf(o[u][h].y, w, acc[h].y);
            acc[h].z = fmaf(o[u][h].z, w, acc[h].z);
            acc[h].w = fmaf(o[u][h].w, w, acc[h].w);
          }
        }
      }
      if (W > 1) {  // join the warps' shares of the parts (block-uniform branch)
        __syncthreads();
        red[warp][0][lane] = acc[0];
        red[warp][1][lane] = acc[1];
        if (lane == 0) red_ml[warp] = make_float2(M, L);
        __syncthreads();
        if (sub == 0) {
          float Mt = M;
          for (int w = 1; w < W; ++w) Mt = fmaxf(Mt, red_ml[warp + w].x);
          const float ref = Mt == -INFINITY ? 0.f : Mt, f = exp2f(M - ref);
          M = Mt;
          L *= f;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            acc[h].x *= f; acc[h].y *= f; acc[h].z *= f; acc[h].w *= f;
          }
          for (int w = 1; w < W; ++w) {
            const float2 ml = red_ml[warp + w];
            const float g2 = exp2f(ml.x - ref);
            L = fmaf(ml.y, g2, L);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const float4 o = red[warp + w][h][lane];
              acc[h].x = fmaf(o.x, g2, acc[h].x);
              acc[h].y = fmaf(o.y, g2, acc[h].y);
              acc[h].z = fmaf(o.z, g2, acc[h].z);
              acc[h].w = fmaf(o.w, g2, acc[h].w);
            }
          }
        }
      }
      if (sub != 0) continue;
      const float inv = 1.f / L;
      const int64_t orow = row0 + row;
      if (a.lse && on0 && e == 0) a.lse[orow] = (M + log2f(L)) * 0.6931471805599453f;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (h == 0 ? !on0 : !on1) continue;
        const int64_t at = orow * a.r + e + 128 * h;
        const float4 v = make_float4(acc[h].x * inv, acc[h].y * inv, acc[h].z * inv, acc[h].w * inv);
        if (a.out_f32 || sizeof(T) == 4)
          *reinterpret_cast<float4*>(reinterpret_cast<float*>(a.out) + at) = v;
        else
          *reinterpret_cast<uint2*>(reinterpret_cast<__nv_bfloat16*>(a.out) + at) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
      }
    }
  }
}

template <typename T>
static auto simt_kernel(int r) -> void (*)(const PagedAttnArgs) {
  if (r <= 64) return paged_attn_simt_kernel<T, 0>;
  if (r <= 128) return paged_attn_simt_kernel<T, 1>;
  if (r <= 256) return paged_attn_simt_kernel<T, 2>;
  return paged_attn_simt_kernel<T, 4>;
}

}  // namespace psimt

int paged_simt_grid(int r, int d_R, int dtype, int sms) {
  // the occupancy of the last widths asked for on this thread (the widest
  // shared memory is allowed once per kernel and device)
  struct Last {
    int dev = -1, r, d_R, dtype, grid;
  };
  thread_local Last last;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (last.dev == dev && last.r == r && last.d_R == d_R && last.dtype == dtype) return last.grid;
  auto k = dtype == MTLA_BF16 ? psimt::simt_kernel<__nv_bfloat16>(r) : psimt::simt_kernel<float>(r);
  int occ = 0;
  if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)psimt::smem_bytes(psimt::MAXD, dtype == MTLA_BF16 ? 2 : 4)) != cudaSuccess)
    return 0;
  if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&occ, k, psimt::NT, psimt::smem_bytes(r + d_R, dtype == MTLA_BF16 ? 2 : 4)) != cudaSuccess ||
      occ < 1)
    return 0;
  last.dev = dev;
  last.r = r;
  last.d_R = d_R;
  last.dtype = dtype;
  last.grid = sms * (occ < 4 ? occ : 4);
  return last.grid;
}

cudaError_t launch_paged_attn_simt(const PagedAttnArgs& a, int grid, int dtype, cudaStream_t st) {
  auto k = dtype == MTLA_BF16 ? psimt::simt_kernel<__nv_bfloat16>(a.r) : psimt::simt_kernel<float>(a.r);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(psimt::NT);
  cfg.dynamicSmemBytes = psimt::smem_bytes(a.r + a.d_R, dtype == MTLA_BF16 ? 2 : 4);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k, a);
}

cudaError_t launch_paged_combine(const PagedAttnArgs& a, int grid, int sms, int dtype, cudaStream_t st) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  // As many blocks as are resident at once, up to one a row (of the average
  // sequence's items).  An x for every block of the attention; where those leave
  // too few y and items are far fewer, one for every item, which it then has to
  // look for (fp32 chunks, up to 41 items in 296 blocks: the joining 6.6 -> 3.3 us;
  // 32 decode tokens in 148 blocks would take 1 us more).
  const int64_t items = (a.c.N + a.plan.tpt - 1) / a.plan.tpt + a.c.B, most = items < a.c.N ? items : a.c.N;
  const int64_t item = (a.c.N + (int64_t)a.c.B - 1) / a.c.B * a.H, rows = item < a.rows ? item : a.rows;
  const int64_t fit = 8 * (int64_t)sms;
  const bool seek = fit / grid < rows && 4 * most <= grid;
  const int64_t gx = seek ? most : grid, y = fit / gx < 1 ? 1 : (fit / gx < rows ? fit / gx : rows);
  cfg.gridDim = dim3((unsigned)gx, (unsigned)y);
  cfg.blockDim = dim3(psimt::CNT);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return dtype == MTLA_BF16 ? cudaLaunchKernelEx(&cfg, psimt::paged_combine_kernel<__nv_bfloat16>, a, seek ? grid : 0)
                            : cudaLaunchKernelEx(&cfg, psimt::paged_combine_kernel<float>, a, seek ? grid : 0);
}

}  // namespace mtla
