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
//  * Two metadata warps work a tile ahead: they find the tokens' sequences and
//    leave P rows, pool rows, positions and bit masks (which tokens open a
//    group, end a chunk, ...) in shared memory, and send the tile's P rows
//    towards L2.  The epilogue's 12 warps take 32 columns each in chunks of 8
//    (8 prompt chunks, 23,000 tokens, s = 2: 32.2 us, 1.87 TB/s of what has to
//    move; of 16 columns 33.0, whose longer code misses the instruction cache
//    more; of 4 35.2).  They are bound by issue and by the latency of their
//    chain, so P comes to shared memory by asynchronous copies while the tile
//    before is stored, and finished rows leave through a staging block, 16 bytes
//    of eight rows a step.
//  * RoPE: an exact angle every 8 tokens of a run of positions and a rotation
//    by the pair's own angle between them (at most seven single-precision
//    products: error below 2^-20 of the key).  Where the exact angles lie follows
//    the tile's columns, so a token's RoPE channels keep that bound but not their
//    last bits when its chunk is cut elsewhere; its latent channels' entries and
//    sums are the same bits in every cut.  (An angle that depends on the position
//    alone, an exact one at every 8th or 32nd position and a table of the turns
//    between, took 33.2 and 34.5 us for the 23,000 tokens.)
//  * The queries are a stream of their own (no tile needs them): a second,
//    small kernel rotates them on the registers that this one leaves free, on
//    the same SMs at the same time.
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
constexpr int NPART = NWARPS / 4, PCOL = NTOK / NPART;  // column parts of a tile (4) and their columns (32)
constexpr int CH = 8;                          // columns of a chunk
constexpr int NEPI = 3 * NPART;                // epilogue warps
constexpr int TMA_WARP = 3, MMA_WARP = 7, META_WARP0 = 11, META_WARP1 = 15;  // warps of the padding quarter
constexpr uint32_t TMEM_COLS = 512, ACC_STRIDE = 128, HI_COL = 256, LO_COL = 384;
constexpr uint32_t IDESC = umma_idesc_bf16(M, NTOK, false, false);

// What the epilogue needs to know of a tile's tokens.
struct Meta {
  int prow[NTOK];       // P row
  int pool[NTOK];       // pool row of a token that writes one
  uint32_t pos[NTOK];   // position (0-based time)
  int seq[NTOK];
  int back[NTOK];       // tokens of its group in the chunk before it
  uint32_t taken[4];    // bit l of word m: token 32 m + l.  A sequence takes it
  uint32_t open[4];     // the sum starts here (with a carry: at tail_in)
  uint32_t carry[4];
  uint32_t last[4];     // last token of its chunk
  uint32_t row[4];      // it writes a cache row
  uint32_t turn[4];     // its position is not the previous token's plus one
};

constexpr size_t OFF_B = 0;
constexpr size_t OFF_KR = OFF_B + (size_t)KS * BBLK;
constexpr size_t OFF_META = OFF_KR + 2 * (size_t)KRBLK;
constexpr size_t OFF_OST = (OFF_META + 2 * sizeof(Meta) + 127) / 128 * 128;  // staged rows: 2 KB an epilogue warp
constexpr size_t OFF_P = OFF_OST + (size_t)NEPI * PCOL * 64;  // P of a tile: 32 columns x 32 channels a warp, fp32
constexpr size_t OFF_ROPE = OFF_P + (size_t)NEPI * PCOL * 128;
constexpr size_t OFF_BAR = OFF_ROPE + (DR / 2) * 8;
constexpr int NBAR = 2 * KS + 2 * 4 + 1;
constexpr size_t OFF_TMEM = OFF_BAR + NBAR * 8;
constexpr size_t SMEM = OFF_TMEM + 16 + 1024;
static_assert(SMEM <= 232448, "one block's shared memory (227 KB)");
static_assert(OFF_ROPE % 8 == 0 && sizeof(Meta) % 16 == 0 && OFF_META % 16 == 0 && OFF_BAR % 8 == 0, "alignment");

__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity));
}
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
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
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(__fadd_rn(1.f, e)));
  return __fmul_rn(v, r);  // (rounded by itself, as in gated2)
}
// The same for two columns, y = (g + bc) p: sums and products two an instruction
// (packed fp32).
__device__ __forceinline__ void gated2(float& v0, float& v1, uint32_t g0, uint32_t g1, float bc, float p0, float p1) {
  asm("{\n .reg .b64 g, b, p, v, o;\n .reg .f32 x, y;\n"
      " mov.b64 g, {%2, %3};\n mov.b64 b, {%4, %4};\n mov.b64 p, {%5, %6};\n mov.b64 v, {%0, %1};\n"
      " add.rn.f32x2 g, g, b;\n mul.rn.f32x2 g, g, p;\n"
      " mov.b64 {x, y}, g;\n ex2.approx.ftz.f32 x, x;\n ex2.approx.ftz.f32 y, y;\n mov.b64 g, {x, y};\n"
      " mov.b64 o, {0f3F800000, 0f3F800000};\n add.rn.f32x2 g, g, o;\n"
      " mov.b64 {x, y}, g;\n rcp.approx.ftz.f32 x, x;\n rcp.approx.ftz.f32 y, y;\n mov.b64 g, {x, y};\n"
      " mul.rn.f32x2 v, v, g;\n mov.b64 {%0, %1}, v;\n}"
      : "+f"(v0), "+f"(v1) : "f"(__uint_as_float(g0)), "f"(__uint_as_float(g1)), "f"(bc), "f"(p0), "f"(p1));
}
constexpr float kNegLog2e = -1.4426950408889634f;

// Rotates the queries: a warp takes QROWS token rows (one search for their
// sequences), four a step with the next step's loads in flight; a half of the
// warp computes a token's 16 angles, a lane turns 16 bytes of a row.  It reads
// nothing that the append kernel writes, so it starts as soon as that one has
// started (by then everything before both is complete) and waits for it only
// at its end, so that what follows finds both done.
constexpr int QROWS = 8, QT = 256;
__global__ void __launch_bounds__(QT, 4) paged_rotate_kernel(const __grid_constant__ PagedAppendArgs a) {
  const int lane = threadIdx.x & 31, words = a.H * (DR / 8);
  const int64_t i = ((int64_t)blockIdx.x * (QT / 32) + (threadIdx.x >> 5)) * QROWS;
  if (i < a.c.N) {
    const uint4* src = reinterpret_cast<const uint4*>(a.q_rope);
    uint4* dst = reinterpret_cast<uint4*>(a.q_rope_out);
    const uint64_t turn = a.rotate ? a.rope.turns[lane & 15] : 0;
    int b;
    AppendWin w;
    warp_windows(a, i, b, w);
    const int64_t place = i + lane - w.first;
    const uint32_t taken =
        __ballot_sync(0xffffffffu, lane < QROWS && i + lane < a.c.N && b >= 0 && place >= 0 && place < w.n);
    const uint32_t pos = (uint32_t)w.t0 + (uint32_t)place;
#pragma unroll 1
    for (int word = lane; word < (words + 31) / 32 * 32; word += 32) {
      uint4 v[4], next[4];
      auto load = [&](uint4 (&x)[4], int k) {
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          x[h] = make_uint4(0, 0, 0, 0);
          if ((taken >> (k + h) & 1) && word < words) x[h] = src[(i + k + h) * words + word];
        }
      };
      load(next, 0);
#pragma unroll 1
      for (int k = 0; k < QROWS; k += 4) {
#pragma unroll
        for (int h = 0; h < 4; ++h) v[h] = next[h];
        if (k + 4 < QROWS) load(next, k + 4);
#pragma unroll
        for (int g = 0; g < 4; g += 2) {
          const float2 cs = rope_cos_sin(__shfl_sync(0xffffffffu, pos, k + g + (lane >> 4)), turn);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t x[4] = {v[g + h].x, v[g + h].y, v[g + h].z, v[g + h].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {        // pair 4 (word mod 4) + e
              const int sl = 16 * h + 4 * (word & 3) + e;
              const float co = __shfl_sync(0xffffffffu, cs.x, sl), si = __shfl_sync(0xffffffffu, cs.y, sl);
              const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&x[e]));
              x[e] = pack_bf16x2(f.x * co - f.y * si, f.x * si + f.y * co);
            }
            if ((taken >> (k + g + h) & 1) && word < words)
              dst[(i + k + g + h) * words + word] = make_uint4(x[0], x[1], x[2], x[3]);
          }
        }
      }
    }
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

__global__ void __maxnreg__(96) paged_append_tc_kernel(const __grid_constant__ PagedAppendMaps mp,
                                                                const __grid_constant__ PagedAppendArgs a, int n_tiles, int cols) {
  extern __shared__ uint8_t smem_raw[];
  // (an offset, not an integer address: the compiler keeps seeing shared memory)
  uint8_t* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint64_t* bar = reinterpret_cast<uint64_t*>(sm + OFF_BAR);
  uint64_t* const k_full = bar;                  // [KS]
  uint64_t* const k_empty = bar + KS;            // [2] a tile's stages (epilogue)
  uint64_t* const acc_full = bar + 2 * KS;       // [2]
  uint64_t* const acc_empty = acc_full + 2;      // [2]
  uint64_t* const meta_full = acc_full + 4;      // [2]
  uint64_t* const meta_empty = acc_full + 6;     // [2]
  uint64_t* const mma_done = acc_full + 8;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(sm + OFF_TMEM);
  Meta* meta = reinterpret_cast<Meta*>(sm + OFF_META);
  uint64_t* turns = reinterpret_cast<uint64_t*>(sm + OFF_ROPE);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int ct = blockIdx.x % CT, G = gridDim.x / CT, j0 = blockIdx.x / CT;
  const int u_beg = (int)((int64_t)j0 * n_tiles / G), u_end = (int)((int64_t)(j0 + 1) * n_tiles / G);
  const bool has_rope = (ct + 1) * NCT > R;
  const int s = a.s, halo = s - 1, nout = cols - halo;  // columns in use; tokens of a tile
  const int q = warp & 3, part = warp >> 2;      // TMEM lane quarter; quarter of the tile's columns
  const bool epi = q < 3;
  const int ch = ct * NCT + q * 32 + lane;       // this thread's channel (epilogue warps)

  if (tid == 0) {
    for (int i = 0; i < KS; ++i) {
      mbar_init(&k_full[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&k_empty[i], NEPI);
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], NEPI);
      mbar_init(&meta_full[i], 2);
      mbar_init(&meta_empty[i], NEPI);
    }
    mbar_init(mma_done, 1);
    fence_mbar_init();
  }
  if (tid < DR / 2) turns[tid] = a.rotate ? a.rope.turns[tid] : 0;  // (no rotation: by nothing)
  if (warp == 0) {
    tmem_alloc(tmem_holder, TMEM_COLS);
    tmem_relinquish();
  }
  if (warp == TMA_WARP && lane == 0) {
    prefetch_tmap(&mp.c);
    prefetch_tmap(&mp.kr);
  }
  // (the query kernel may start once all before this call is complete)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // W_c^T: all of its loads in flight before anything else
  float wv[64];
  if (epi) {
#pragma unroll
    for (int k = 0; k < 64; ++k) wv[k] = __ldg(a.m.W_c + (size_t)(64 * part + k) * D + ch);
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
        const int b2 = (u - u_beg) & 1;
        if (u - u_beg >= 2 && !mbar_wait(&k_empty[b2], (((u - u_beg) >> 1) & 1) ^ 1)) { ok = false; break; }
        for (int kb = 0; kb < KB; ++kb, ++kc) {
          const int st = kc % KS;
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
  } else if (warp == META_WARP0 || warp == META_WARP1) {
    // ======================= token metadata, one tile ahead: 64 tokens a warp =======================
    const int m0 = warp == META_WARP0 ? 0 : 2;
    uint32_t tc = 0;
    for (int u = u_beg; u < u_end; ++u, ++tc) {
      const int mb = tc & 1;
      const int64_t base = (int64_t)u * nout - halo;
      int b[2];
      warp_sequences<2>(a.c, base + 32 * m0, b);
      // windows of both tokens of a lane, then their table entries: two
      // round trips a tile
      AppendWin w[2];
#pragma unroll
      for (int m = 0; m < 2; ++m) w[m] = seq_win(a.c, b[m] < 0 ? 0 : b[m]);
      uint32_t pos[2], grp[2];
      int back[2];
      uint32_t fl[2];
      const int32_t* entry[2];
      int slot[2];
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        append_fit(a, w[m], false);
        const int64_t i = base + lane + 32 * (m0 + m), place = i - w[m].first;
        const bool taken = b[m] >= 0 && i >= 0 && place >= 0 && place < w[m].n;
        const uint32_t tm = taken ? (uint32_t)w[m].t0 + (uint32_t)place : 0;  // 0-based time
        const uint32_t g = div32(tm, a.div_s), in = tm - g * (uint32_t)s;
        const bool last = taken && place + 1 == w[m].n;
        pos[m] = tm;
        grp[m] = g;
        back[m] = taken ? (int)(in < place ? (int64_t)in : place) : 0;
        const bool row = taken && (last || in + 1 == (uint32_t)s) && lane + 32 * (m0 + m) >= halo;
        fl[m] = (taken ? 1u : 0u) | (taken && (in == 0 || place == 0) ? 2u : 0u) | (taken && in != 0 && place == 0 ? 4u : 0u) |
                (last ? 8u : 0u) | (row ? 16u : 0u);
        const uint32_t k = div32(g, a.p.div_rows);
        entry[m] = row ? a.p.table + (int64_t)b[m] * a.p.table_pages + k : nullptr;
        slot[m] = (int)(g - k * (uint32_t)a.p.page_rows);
      }
      // the tile's P rows (this CTA's channels) towards L2, a tile ahead of their use
#pragma unroll
      for (int m = 0; m < 2; ++m)
        if ((fl[m] & 3) == 3 || (fl[m] & 1 && lane + 32 * (m0 + m) == 0)) {
          const float* row = a.m.P + (int64_t)grp[m] * D + ct * NCT;
#pragma unroll
          for (int k = 0; k < 3; ++k) asm volatile("prefetch.global.L2 [%0];" ::"l"(row + 32 * k));
        }
      int32_t page[2];
#pragma unroll
      for (int m = 0; m < 2; ++m) page[m] = entry[m] ? *entry[m] : -1;
      if (tc >= 2 && !warp_wait(&meta_empty[mb], ((tc >> 1) & 1) ^ 1)) { ok = false; break; }
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        const bool in_pool = page[m] >= 0 && page[m] < a.p.num_pages;
        if (entry[m] && !in_pool) set_err(a.dev_err, MTLA_DEVERR_CAPACITY);
        Meta& mt = meta[mb];
        mt.prow[lane + 32 * (m0 + m)] = (int)grp[m];
        mt.pool[lane + 32 * (m0 + m)] = in_pool ? page[m] * a.p.page_rows + slot[m] : -1;
        mt.pos[lane + 32 * (m0 + m)] = pos[m];
        mt.seq[lane + 32 * (m0 + m)] = b[m];
        mt.back[lane + 32 * (m0 + m)] = back[m];
        const uint32_t taken = __ballot_sync(0xffffffffu, fl[m] & 1), open = __ballot_sync(0xffffffffu, fl[m] & 2),
                       carry = __ballot_sync(0xffffffffu, fl[m] & 4), last = __ballot_sync(0xffffffffu, fl[m] & 8),
                       row = __ballot_sync(0xffffffffu, in_pool);
        const uint32_t before = __shfl_up_sync(0xffffffffu, pos[m], 1);
        const uint32_t turn = __ballot_sync(0xffffffffu, lane == 0 || pos[m] != before + 1);
        if (lane == 0) {
          meta[mb].taken[m0 + m] = taken;
          meta[mb].open[m0 + m] = open;
          meta[mb].carry[m0 + m] = carry;
          meta[mb].last[m0 + m] = last;
          meta[mb].row[m0 + m] = row;
          meta[mb].turn[m0 + m] = turn;
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&meta_full[mb]);
    }
    if (!ok && lane == 0) set_err(a.dev_err, MTLA_DEVERR_TIMEOUT);
    if (warp == META_WARP1)                      // per-sequence results, a lane each
      for (int b0 = blockIdx.x * 32; b0 < a.c.B; b0 += gridDim.x * 32) {
        const int b = b0 + lane;
        bool copy = false;
        if (b < a.c.B) {
          const AppendWin w = append_win(a, b, true);
          a.t_out[b] = (int32_t)(w.t0 + w.n);
          if (a.cache_len) a.cache_len[b] = w.t0 + w.n > 0 ? (int32_t)group_of(w.t0 + w.n, s) : 0;
          copy = w.n == 0;
        }
        for (uint32_t left = __ballot_sync(0xffffffffu, copy); left; left &= left - 1) {
          const int64_t row = (int64_t)(b0 + __ffs(left) - 1) * D;
          for (int k = lane; k < D; k += 32) a.tail_out[row + k] = a.tail_in[row + k];
        }
      }
    if (!ok && lane == 0) set_err(a.dev_err, MTLA_DEVERR_TIMEOUT);
  } else {
    // ======================= epilogue warps =======================
    const bool rope = ch >= R;                   // warp-uniform
    const uint32_t lane_base = tmem + ((uint32_t)(q * 32) << 16);
    {
      // -log2(e) W^T as two bf16 parts into TMEM (loads issued at the kernel's
      // start): the accumulator and the bias are then the base-2 exponent's
      uint32_t hi[32], lo[32];
#pragma unroll
      for (int k = 0; k < 32; ++k) {
        const float w0 = wv[2 * k] * kNegLog2e, w1 = wv[2 * k + 1] * kNegLog2e;
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
    const float bc = __ldg(a.m.b_c + ch) * kNegLog2e;
    const float* Pc = a.m.P + ch;
    const uint32_t sB = smem_u32(sm + OFF_B);
    // this channel's byte inside a swizzled 128-byte latent row (K block ch / 64)
    const uint32_t c_kb = (uint32_t)((ch & 255) >> 6), c_chunk = (uint32_t)((ch & 63) >> 3), c_in = (uint32_t)(ch & 7) * 2;
    uint32_t xo[8];                              // byte of the channel's 16-byte piece in row r of a swizzle atom
#pragma unroll
    for (int r = 0; r < 8; ++r) xo[r] = (c_chunk ^ (uint32_t)r) << 4;
    // staged rows: [PCOL columns][32 channels] bf16, read back in 16-byte pieces
    uint8_t* const ost = sm + OFF_OST + (part * 3 + q) * (PCOL * 64);
    const uint32_t ost_ch = smem_u32(ost) + lane * 2;
    const int ch0 = ct * NCT + q * 32;           // the warp's first channel
    const uint64_t turn = turns[lane >> 1];      // (rope quarter) the channel's pair
    const float2 step = rope_cos_sin(1, turn);
    auto turned = [&](uint32_t pair, float2 cs) -> float {
      const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&pair));
      return ch & 1 ? f.y * cs.x + f.x * cs.y : f.x * cs.x - f.y * cs.y;
    };
    // P of a tile's columns [p0, p0 + PCOL), this warp's channels, into its
    // block of shared memory by asynchronous copies: issued while the tile
    // before is stored (a copy a column: the same row again is an L1 hit)
    const int p0 = PCOL * part;
    const uint32_t pbuf = smem_u32(sm + OFF_P + (size_t)(part * 3 + q) * (PCOL * 128)) + lane * 4;
    auto fetch = [&](const Meta& mt) {
#pragma unroll 2
      for (int k = 0; k < PCOL; k += 4) {
        const int4 r = *reinterpret_cast<const int4*>(&mt.prow[p0 + k]);
        const int rows[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(pbuf + (k + e) * 128), "l"(Pc + (int64_t)rows[e] * D)
                       : "memory");
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    ok = warp_wait(&meta_full[0], 0);
    if (ok) fetch(meta[0]);
    uint32_t tc = 0;
    for (int u = u_beg; u < u_end && ok; ++u, ++tc) {
      const int ab = tc & 1, sb = ab * KB;
      const uint32_t par = (tc >> 1) & 1;
      const int64_t base = (int64_t)u * nout - halo;
      const Meta& mt = meta[ab];
      // this warp's columns [cb, ce) of [p0, p0 + PCOL); masks are bits of the column in its word of 32
      const int cb = p0 > halo ? p0 : halo;
      const int64_t lastc = a.c.N - base < cols ? a.c.N - base : cols;  // columns past it are no token rows, or the next tile's
      const int ce = p0 + PCOL < lastc ? p0 + PCOL : (int)lastc;
      if (cb < ce) {
        const uint32_t vrow = rope ? smem_u32(sm + OFF_KR + ab * KRBLK) + (uint32_t)(lane >> 1) * 4 : sB + (sb + c_kb) * BBLK + c_in;
        // Columns before cb belong to a group that began before them: it is
        // summed again from its start in the chunk.  A few of them singly (same
        // P, and the tail if that start is the chunk's), more in chunks of 8.
        const int back = mt.back[cb], c1 = cb - back;
        const bool single = back > 0 && back < 8 && cb == p0;
        const int c_beg = single ? p0 : c1 & ~(CH - 1);
        float ph = 0.f, run = 0.f;
        if (single) {
          ph = __ldg(Pc + (int64_t)mt.prow[cb] * D);
          if (mt.carry[c1 >> 5] >> (c1 & 31) & 1) run = a.tail_in[(int64_t)mt.seq[cb] * D + ch];
        }
        ok = warp_wait(&acc_full[ab], par) && warp_wait(&k_full[sb], par) && warp_wait(&k_full[sb + c_kb], par);
        tc_fence_after();
        if (!ok) break;
        const uint32_t acc = lane_base + ab * ACC_STRIDE;
        if (single) {
#pragma unroll 1
          for (int col = c1; col < cb; ++col) {
            const uint32_t g = tmem_ld1(acc + col);
            float x;
            if (rope) {
              uint32_t pair;
              asm volatile("ld.shared.u32 %0, [%1];" : "=r"(pair) : "r"(vrow + (uint32_t)col * (DR * 2)));
              x = turned(pair, rope_cos_sin(mt.pos[col], turn));
            } else {
              uint16_t raw;
              asm volatile("ld.shared.u16 %0, [%1];" : "=h"(raw) : "r"(vrow + (uint32_t)(col >> 3) * 1024 + (uint32_t)(col & 7) * 128 +
                                                                       ((c_chunk ^ (uint32_t)(col & 7)) << 4)));
              x = __bfloat162float(__ushort_as_bfloat16(raw));
            }
            tmem_wait_ld();
            run = __fadd_rn(run, gated(x, __fmul_rn(__fadd_rn(__uint_as_float(g), bc), ph)));
          }
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
#pragma unroll 1
        for (int c0 = c_beg; c0 < ce; c0 += CH) {
          uint32_t g[CH];
          tmem_ld8(acc + c0, g);
          const int word = c0 >> 5, bit = c0 & 31;
          float v[CH], pc[CH];
          if (c0 >= p0) {
#pragma unroll
            for (int k = 0; k < CH; ++k) asm volatile("ld.shared.f32 %0, [%1];" : "=f"(pc[k]) : "r"(pbuf + (c0 - p0 + k) * 128));
          } else {
#pragma unroll
            for (int k = 0; k < CH; ++k) pc[k] = __ldg(Pc + (int64_t)mt.prow[c0 + k] * D);
          }
          if (rope) {
            const uint32_t at = vrow + (uint32_t)c0 * (DR * 2);
            uint32_t pair[CH];
#pragma unroll
            for (int k = 0; k < CH; ++k) asm volatile("ld.shared.u32 %0, [%1];" : "=r"(pair[k]) : "r"(at + k * (DR * 2)));
            if ((mt.turn[word] >> bit & 0xfeu) == 0) {  // one run of positions
              const uint32_t first = mt.pos[c0];
              float2 cs = make_float2(1.f, 0.f);
#pragma unroll
              for (int k = 0; k < CH; ++k) {
                cs = (k & 7) == 0 ? rope_cos_sin(first + k, turn)
                                  : make_float2(cs.x * step.x - cs.y * step.y, cs.x * step.y + cs.y * step.x);
                v[k] = turned(pair[k], cs);
              }
            } else {
#pragma unroll
              for (int k = 0; k < CH; ++k) v[k] = turned(pair[k], rope_cos_sin(mt.pos[c0 + k], turn));
            }
          } else {
            const uint32_t at = vrow + (uint32_t)(c0 >> 3) * 1024;
#pragma unroll
            for (int k = 0; k < CH; ++k) {
              uint16_t raw;
              asm volatile("ld.shared.u16 %0, [%1];" : "=h"(raw) : "r"(at + (k >> 3) * 1024 + (k & 7) * 128 + xo[k & 7]));
              v[k] = __bfloat162float(__ushort_as_bfloat16(raw));
            }
          }
          tmem_wait_ld();
#pragma unroll
          for (int k = 0; k < CH; k += 2) gated2(v[k], v[k + 1], g[k], g[k + 1], bc, pc[k], pc[k + 1]);
          // the sums, in token order (what a column before the first open group
          // holds is never stored); a chunk that goes on in an open group starts
          // at its tail
          const uint32_t open = mt.open[word] >> bit, carry = mt.carry[word] >> bit & 0xffu;
          if (carry) {
#pragma unroll
            for (int k = 0; k < CH; ++k)
              if (carry >> k & 1) v[k] += a.tail_in[(int64_t)mt.seq[c0 + k] * D + ch];
          }
#pragma unroll
          for (int k = 0; k < CH; ++k) {
            run = (open >> k & 1 ? 0.f : run) + v[k];
            v[k] = run;
          }
          if (c0 >= p0) {
            const uint32_t last = mt.last[word] >> bit & 0xffu;
            if (last) {
#pragma unroll
              for (int k = 0; k < CH; ++k)
                if ((last >> k & 1) && c0 + k >= cb && c0 + k < ce) a.tail_out[(int64_t)mt.seq[c0 + k] * D + ch] = v[k];
            }
            const uint32_t at = ost_ch + (uint32_t)(c0 - p0) * 64;
#pragma unroll
            for (int k = 0; k < CH; k += 2) {
              const uint32_t w = pack_bf16x2(v[k], v[k + 1]);
              asm volatile("st.shared.u16 [%0], %1;" ::"r"(at + k * 64), "h"((uint16_t)(w & 0xffffu)) : "memory");
              asm volatile("st.shared.u16 [%0], %1;" ::"r"(at + k * 64 + 64), "h"((uint16_t)(w >> 16)) : "memory");
            }
          }
        }
        if (u + 1 < u_end) {
          if (!warp_wait(&meta_full[ab ^ 1], ((tc + 1) >> 1) & 1)) { ok = false; break; }
          fetch(meta[ab ^ 1]);
        }
        // the staged rows, 16 bytes of eight rows a step
        __syncwarp();
        const uint32_t taken = a.row_state ? mt.taken[p0 >> 5] : 0u, rows = mt.row[p0 >> 5];
        const int piece = lane & 3;
#pragma unroll
        for (int k8 = 0; k8 < PCOL / 8; ++k8) {
          const int r = 8 * k8 + (lane >> 2), col = p0 + r, bit = col & 31;
          const uint4 w = *reinterpret_cast<const uint4*>(ost + r * 64 + piece * 16);
          if (col >= cb && col < ce) {
            if (taken >> bit & 1)
              *reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(a.row_state) + (base + col) * D + ch0 + piece * 8) = w;
            if (rows >> bit & 1)
              *reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(a.p.pages) + (int64_t)mt.pool[col] * a.p.row_stride +
                                        ch0 + piece * 8) = w;
          }
        }
      } else if (u + 1 < u_end) {
        if (!warp_wait(&meta_full[ab ^ 1], ((tc + 1) >> 1) & 1)) { ok = false; break; }
        fetch(meta[ab ^ 1]);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&acc_empty[ab]);
        mbar_arrive(&meta_empty[ab]);
        mbar_arrive(&k_empty[ab]);
      }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");  // no copy may still be writing shared memory at exit
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
  static std::atomic<uint64_t> done_mask{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !(done_mask & (1ull << dev))) {
    e = cudaFuncSetAttribute(ptp::paged_append_tc_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)ptp::SMEM);
    if (e != cudaSuccess) return e;
    // the same shared-memory configuration for both kernels: they share SMs
    e = cudaFuncSetAttribute(ptp::paged_append_tc_kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                             cudaSharedmemCarveoutMaxShared);
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(ptp::paged_rotate_kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                             cudaSharedmemCarveoutMaxShared);
    if (e != cudaSuccess) return e;
    if (dev < 64) done_mask |= 1ull << dev;
  }
  int per = sms / ptp::CT > 0 ? sms / ptp::CT : 1;  // CTAs per channel tile
  // The fewest columns (a warp's part each) that give no CTA a second tile, unless
  // the first s - 1 would be half of them: a scheduler then serves fewer warps
  // (four tokens of 128 sequences 13.0 us, with 128 columns 15.3; one of 512
  // 15.6 / 18.0; one sequence of 1024 10.5 / 11.2).
  int cols = ptp::PCOL;
  while (cols < ptp::NTOK && (cols < 2 * (a.s - 1) || cdiv(a.c.N, cols - (a.s - 1)) > per)) cols += ptp::PCOL;
  const int n_tiles = (int)cdiv(a.c.N, cols - (a.s - 1));
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
  e = cudaLaunchKernelEx(&cfg, ptp::paged_append_tc_kernel, m, a, n_tiles, cols);
  if (e != cudaSuccess || !a.q_rope) return e;
  cfg.gridDim = dim3((unsigned)cdiv(a.c.N, ptp::QT / 32 * ptp::QROWS));
  cfg.blockDim = dim3(ptp::QT);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, ptp::paged_rotate_kernel, a);
}

}  // namespace mtla
