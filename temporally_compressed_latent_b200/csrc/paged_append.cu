// Appending a chunk of new tokens to a paged cache: the generic kernel (any
// supported dims, fp32 or bf16 storage, fp32 arithmetic).
//
// What it computes (MTLA paper notes, "Key designs: hyper-network temporal
// merging"): for every token, the gate w = sigmoid((c W_c + b_c) * P[j-1]), the
// gated entry e = w * [c ; k^R] with k^R rotated to the token's position, and
// the running sum of its group, S_t = S_{t-1} + e.
//
// The tokens of all sequences lie one after another in the token arrays, so a
// block takes a tile of consecutive token rows whatever sequences they belong
// to, and 32 of the row's D channels.  Its 256 threads split the r latents of
// the gate contraction eight ways; a thread keeps its 1/8 of a channel's
// column of W_c in registers for the whole tile, so W_c is read once a block.
// A tile that begins inside a group recomputes the entries of the group's
// earlier tokens (at most s - 1), so that no block waits for another; the sums
// run from the group's start in token order in every tile, which makes them
// independent of the tiling: one call or several give the same bits.
//
// Few tokens: the chain of dependent reads bounds it.  So W_c, the latents of
// the first round (with a short stride the rows before a tile are taken
// whether needed or not, and no read waits to know) and the sequences' windows
// are all requested at the start, and P, the tails, the RoPE keys and the table
// entries as soon as the windows are known, before the products.  One token takes
// 4.4 us (of which a launch is 2 to 3), one token of 32 sequences 5.5 us, 24 fp32
// sequences of 5 drafts 4.1 us.
#include "paged.cuh"

namespace mtla {
namespace pap {

constexpr int NT = 256, NW = NT / 32;
constexpr int U = 16;                // tokens of one round
constexpr int RESIDENT = 2;          // blocks an SM

__device__ __forceinline__ float4 ld4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 ld4(const __nv_bfloat16* p) {
  const uint2 x = *reinterpret_cast<const uint2*>(p);
  const float2 a = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&x.x));
  const float2 b = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&x.y));
  return make_float4(a.x, a.y, b.x, b.y);
}

// One token's place, as the block's threads share it.
struct Tok {
  uint32_t group, pos;  // 0-based group and time
  int seq;              // -1: no sequence takes this row
  uint8_t opens;        // the running sum starts at this token's entry
  uint8_t carry;        // ... with tail_in added
  uint8_t last;         // last token of its sequence's chunk
  uint8_t row;          // it writes a cache row
};

struct alignas(16) Smem {
  float part[NW][U][32];
  float v[U][32];       // gated entries, then sums
  Tok tok[U];
  int64_t i0;
};
static_assert(sizeof(Smem) % 16 == 0 && sizeof(Tok) == 16, "the latents behind it are read four at a time");

// KPT: latents per warp, at least r / 8
template <typename T, int KPT>
__global__ void __launch_bounds__(NT) paged_append_kernel(const __grid_constant__ PagedAppendArgs a, int gate_blocks,
                                                          int rot_blocks) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int D = a.r + a.d_R, s = a.s;

  if ((int)blockIdx.x >= gate_blocks + rot_blocks) {
    // ---- per-sequence results: one warp a sequence
    const int b = (blockIdx.x - gate_blocks - rot_blocks) * NW + warp;
    if (b >= a.c.B) return;
    const AppendWin w = append_win(a, b, lane == 0);
    if (lane == 0) {
      a.t_out[b] = (int32_t)(w.t0 + w.n);
      if (a.cache_len) a.cache_len[b] = w.t0 + w.n > 0 ? (int32_t)group_of(w.t0 + w.n, s) : 0;
    }
    if (w.n == 0)
      for (int k = lane; k < D; k += 32) a.tail_out[(int64_t)b * D + k] = a.tail_in[(int64_t)b * D + k];
    return;
  }
  if ((int)blockIdx.x >= gate_blocks) {
    // ---- RoPE queries: one warp a token, its d_R / 2 angles once for all heads
    const int i = (blockIdx.x - gate_blocks) * NW + warp;
    if (i >= a.c.N) return;
    int b;
    AppendWin w;
    warp_windows(a, i, b, w);
    b = __shfl_sync(0xffffffffu, b, 0);
    w.first = __shfl_sync(0xffffffffu, w.first, 0);
    w.n = __shfl_sync(0xffffffffu, w.n, 0);
    w.t0 = __shfl_sync(0xffffffffu, w.t0, 0);
    if (b < 0 || i < w.first || i - w.first >= w.n) return;
    const uint32_t pos = (uint32_t)(w.t0 + (i - w.first));
    const T* src = reinterpret_cast<const T*>(a.q_rope) + (int64_t)i * a.H * a.d_R;
    T* dst = reinterpret_cast<T*>(a.q_rope_out) + (int64_t)i * a.H * a.d_R;
    const int pairs = a.d_R / 2;
    // a lane's pairs: k, k + 32, ... of all heads in a row
    for (int e = lane; e < a.H * pairs; e += 32) {
      const float x0 = ld_f32(src + 2 * e), x1 = ld_f32(src + 2 * e + 1);
      const float2 cs = a.rotate ? rope_cos_sin(pos, a.rope.turns[e % pairs]) : make_float2(1.f, 0.f);
      st_elem(dst + 2 * e, x0 * cs.x - x1 * cs.y);
      st_elem(dst + 2 * e + 1, x0 * cs.y + x1 * cs.x);
    }
    return;
  }

  Smem& sm = *reinterpret_cast<Smem*>(smem_raw);
  float* cs = reinterpret_cast<float*>(smem_raw + sizeof(Smem));  // [U][8 KPT] latents of the round
  const int slabs = (D + 31) / 32;
  const int ch = (blockIdx.x % slabs) * 32 + lane;   // this thread's channel
  const bool live = ch < D;
  const int64_t i_beg = (int64_t)(blockIdx.x / slabs) * a.tt;
  const int64_t i_end = i_beg + a.tt < a.c.N ? i_beg + a.tt : a.c.N;
  float wv[KPT];
#pragma unroll
  for (int k = 0; k < KPT; ++k) {
    const int kk = warp * KPT + k;
    wv[k] = live && kk < a.r ? __ldg(a.m.W_c + (int64_t)kk * D + ch) : 0.f;
  }
  const float bc = live ? __ldg(a.m.b_c + ch) : 0.f;

  // the first token row: before the tile, where its first group may begin
  int64_t i0 = i_beg - a.halo;
  if (a.halo < 0) {
    if (warp == 0) {
      int b;
      AppendWin w;
      warp_windows(a, i_beg, b, w);
      if (lane == 0) {
        const int64_t place = i_beg - w.first;
        int64_t back = 0;
        if (b >= 0 && place >= 0 && place < w.n) {
          const uint32_t t = (uint32_t)(w.t0 + place), in = t - div32(t, a.div_s) * (uint32_t)s;
          back = in < place ? (int64_t)in : place;
        }
        sm.i0 = i_beg - back;
      }
    }
    __syncthreads();
    i0 = sm.i0;
  }
  float run = 0.f;  // (warp 0) the running sum of this thread's channel
  for (int64_t r0 = i0; r0 < i_end; r0 += U) {
    const int nu = i_end - r0 < U ? (int)(i_end - r0) : U;  // tokens of this round
    for (int k = tid; k < nu * (KPT * NW / 4); k += NT) {
      const int u = k / (KPT * NW / 4), e = (k - u * (KPT * NW / 4)) * 4;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r0 + u >= 0 && e < a.r) {
        const T* src = reinterpret_cast<const T*>(a.m.c_new) + (r0 + u) * a.r + e;
        v = ld4(src);
      }
      *reinterpret_cast<float4*>(cs + u * (KPT * NW) + e) = v;
    }
    if (warp == 0) {  // the round's tokens, a lane each
      int b;
      AppendWin w;
      warp_windows(a, r0, b, w);
      const int64_t i = r0 + lane, place = i - w.first;
      Tok t;
      t.seq = -1;
      t.group = t.pos = 0;
      t.opens = t.carry = t.last = t.row = 0;
      if (lane < nu && i >= 0 && b >= 0 && place >= 0 && place < w.n) {
        t.seq = b;
        t.pos = (uint32_t)(w.t0 + place);
        t.group = div32(t.pos, a.div_s);
        const uint32_t in = t.pos - t.group * (uint32_t)s;
        t.opens = in == 0 || place == 0;
        t.carry = in != 0 && place == 0;
        t.last = place + 1 == w.n;
        t.row = t.last || in + 1 == (uint32_t)s;
      }
      if (lane < U) sm.tok[lane] = t;
    }
    __syncthreads();
    // what this warp's two tokens need later, requested before the products
    float pv[U / NW], tv[U / NW], xv[U / NW], yv[U / NW];
    int32_t page[U / NW];
#pragma unroll
    for (int h = 0; h < U / NW; ++h) {
      const int u = warp + h * NW;
      const Tok t = sm.tok[u];
      pv[h] = tv[h] = xv[h] = yv[h] = 0.f;
      page[h] = -1;
      if (t.seq >= 0) {
        if (t.row && r0 + u >= i_beg)
          page[h] = a.p.table[(int64_t)t.seq * a.p.table_pages + div32(t.group, a.p.div_rows)];
        if (live) {
          pv[h] = __ldg(a.m.P + (int64_t)t.group * D + ch);
          if (t.carry) tv[h] = a.tail_in[(int64_t)t.seq * D + ch];
          if (ch >= a.r) {
            const T* kr = reinterpret_cast<const T*>(a.m.kR_new) + (r0 + u) * a.d_R;
            xv[h] = ld_f32(kr + (ch - a.r));
            if (a.rotate) yv[h] = ld_f32(kr + ((ch - a.r) ^ 1));
          }
        }
      }
    }
    {
      float acc[U];
#pragma unroll
      for (int u = 0; u < U; ++u) acc[u] = 0.f;
#pragma unroll
      for (int g = 0; g < U; g += 4) {
        if (g < nu) {  // four tokens at a time: a few tokens do not pay for sixteen
#pragma unroll
          for (int k = 0; k < KPT; k += 4) {
#pragma unroll
            for (int u = g; u < g + 4; ++u) {
              const float4 c4 = *reinterpret_cast<const float4*>(cs + u * (KPT * NW) + warp * KPT + k);
              acc[u] = fmaf(c4.x, wv[k], acc[u]);
              acc[u] = fmaf(c4.y, wv[k + 1], acc[u]);
              acc[u] = fmaf(c4.z, wv[k + 2], acc[u]);
              acc[u] = fmaf(c4.w, wv[k + 3], acc[u]);
            }
          }
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (u < nu) sm.part[warp][u][lane] = acc[u];
    }
    __syncthreads();
#pragma unroll
    for (int h = 0; h < U / NW; ++h) {  // gated entries
      const int u = warp + h * NW;
      const Tok t = sm.tok[u];
      float e = 0.f;
      if (t.seq >= 0 && live) {
        float g = bc;
#pragma unroll
        for (int w = 0; w < NW; ++w) g += sm.part[w][u][lane];
        float x = xv[h];
        if (ch < a.r) {
          x = cs[u * (KPT * NW) + ch];
        } else if (a.rotate) {
          const int k = ch - a.r;
          const float2 r = rope_cos_sin(t.pos, a.rope.turns[k >> 1]);
          x = (k & 1) ? yv[h] * r.y + x * r.x : x * r.x - yv[h] * r.y;
        }
        // (product and sum rounded one by one: the tail added here and the running
        // sum added below give the same bits)
        e = __fadd_rn(tv[h], __fmul_rn(x, sigmoidf_(g * pv[h])));
      }
      sm.v[u][lane] = e;
    }
    __syncthreads();
    if (warp == 0) {  // running sums, in token order
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (u < nu) {
          run = (sm.tok[u].opens ? 0.f : run) + sm.v[u][lane];
          sm.v[u][lane] = run;
        }
      }
    }
    __syncthreads();
#pragma unroll
    for (int h = 0; h < U / NW; ++h) {
      const int u = warp + h * NW;
      const Tok t = sm.tok[u];
      if (t.seq < 0 || r0 + u < i_beg || !live) continue;
      const float v = sm.v[u][lane];
      if (a.row_state) st_elem(reinterpret_cast<T*>(a.row_state) + (r0 + u) * D + ch, v);
      if (t.row) {
        if (page[h] >= 0 && page[h] < a.p.num_pages) {
          const int64_t row = (int64_t)page[h] * a.p.page_rows + (t.group - div32(t.group, a.p.div_rows) * a.p.page_rows);
          st_elem(reinterpret_cast<T*>(a.p.pages) + row * a.p.row_stride + ch, v);
        } else if (lane == 0) {
          set_err(a.dev_err, MTLA_DEVERR_CAPACITY);
        }
      }
      if (t.last) a.tail_out[(int64_t)t.seq * D + ch] = v;
    }
    __syncthreads();
  }
}

template <typename T>
static auto pick(int r) -> void (*)(const PagedAppendArgs, int, int) {
  if (r <= 64) return paged_append_kernel<T, 8>;
  if (r <= 256) return paged_append_kernel<T, 32>;
  return paged_append_kernel<T, 64>;
}

}  // namespace pap

cudaError_t launch_paged_append_simt(PagedAppendArgs& a, int dtype, int sms, cudaStream_t st) {
  const int D = a.r + a.d_R, slabs = (D + 31) / 32;
  // Tile length: one round of 16 tokens while that does not give every SM its
  // eight blocks, then longer (W_c is read once a block); of fewer tokens where all
  // blocks then start at once and no more than two thirds of its rows are those
  // before it (one token of 32 sequences 5.5 us, in rounds of 16 7.6; four tokens
  // of 44 sequences 7.2, of 16 9.1, of 4 in more blocks than start at once 11.0).
  // A stride of up to 9 takes the s - 1 rows before a tile into its rounds; with a
  // longer one the tile is not below the stride, up to 512 tokens, so that it
  // recomputes at most about its own length again.
  int64_t rounds = cdiv((int64_t)a.c.N * slabs, (int64_t)pap::U * sms * 8);
  rounds = rounds < 1 ? 1 : (rounds > 16 ? 16 : rounds);
  int64_t tt = rounds * pap::U;
  if (a.s <= 9) {
    a.halo = a.s - 1;
    if (rounds == 1)
      for (int few = 4; few < pap::U; few += 4)
        if (2 * few >= 3 * a.halo && cdiv(a.c.N, few - a.halo) * slabs <= (int64_t)sms * pap::RESIDENT) {
          tt = few;
          break;
        }
    tt -= a.halo;
  } else {
    a.halo = -1;
    const int64_t up = cdiv(a.s < 512 ? a.s : 512, pap::U) * pap::U;
    if (tt < up) tt = up;
  }
  a.tt = (int)tt;
  const int kpt = a.r <= 64 ? 8 : (a.r <= 256 ? 32 : 64);
  const size_t smem = sizeof(pap::Smem) + (size_t)pap::U * kpt * pap::NW * 4;
  auto k = dtype == MTLA_BF16 ? pap::pick<__nv_bfloat16>(a.r) : pap::pick<float>(a.r);
  {
    // the shared-memory opt-in, once per instance and device
    static std::atomic<uint64_t> done_mask[6] = {};
    const int slot = (dtype == MTLA_BF16 ? 3 : 0) + (kpt == 8 ? 0 : (kpt == 32 ? 1 : 2));
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64 || !(done_mask[slot] & (1ull << dev))) {
      e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
      if (e != cudaSuccess) return e;
      if (dev < 64) done_mask[slot] |= 1ull << dev;
    }
  }
  const int64_t gate = cdiv(a.c.N, tt) * slabs;
  const int64_t rot = a.q_rope ? cdiv(a.c.N, pap::NW) : 0;
  const int64_t seq = cdiv(a.c.B, pap::NW);
  if (gate + rot + seq >= (int64_t(1) << 31)) return cudaErrorInvalidConfiguration;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(gate + rot + seq));
  cfg.blockDim = dim3(pap::NT);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k, (const PagedAppendArgs)a, (int)gate, (int)rot);
}

}  // namespace mtla
