// Attention of a chunk of new tokens over a paged cache on the 5th-generation
// tensor cores (tcgen05 + TMEM): bf16, r = 256, d_R = 32, any H <= 16.
//
// What it computes (MTLA paper notes, "Key designs: stride-aware causal mask"
// and "decoupled RoPE with temporal compression"; Figure 2(c) of the abstract
// page): the query of a token at time t attends the complete groups before its
// own (cache rows 0 .. ceil(t/s) - 2, found through the block table) and its
// own state row; per (token, head) row an online softmax over the columns.
//
// Design (B200):
//  * An M tile is up to 16 consecutive tokens x H heads <= 128 rows (the heads
//    share every key); a key tile is 64 columns.  One kernel serves every
//    chunk: with one token a sequence only H of the 128 MMA rows are live, but
//    a key tile then costs the tensor pipe about 0.6 us where HBM delivers its
//    36 KB to one of 148 SMs in 0.84 us, so the stream still sets the pace; with
//    long chunks all rows are live and the pipe does.
//  * Work: equal shares of all items' key tiles (paged.cuh), one block an SM; a
//    scheduler warp hands the items of the block's share to the other warps
//    through a ring in shared memory, so no warp reads the sequence arrays on
//    its own path.  Parts of items that a share boundary splits go to the
//    workspace in fp32 and a second kernel joins them.
//  * Three key tiles in flight, four where no item has more than 64 live rows and
//    five where none has more than 40 (the queries' groups leave that room).  A
//    stage is free again only after its value MMA, about 2.3 us after it landed
//    (score MMA, softmax, value MMA), so three stages gave 1.07 us a tile to a
//    decode step; 128 sequences of up to 5 tokens and 8 heads took 57.9 us with
//    four and 55.8 with five.
//  * Tiles are lists of 8-row groups: a group is nine [8 x 64 B] planes with the
//    64-byte swizzle (4608 bytes, one TMA box), so a page of any multiple of 8
//    rows feeds a key tile, the operand's 8-row stride is 4608 everywhere, and
//    only the groups that hold live query rows or visible columns are loaded.
//    The tokens' own states are groups too, behind the cache's: a query's own
//    column is one more column of the last tiles, with no path of its own.
//  * A group's rows past the sequence's end may hold anything, NaN included:
//    their scores are replaced by -inf, and the softmax warps write zeros over
//    their latents once the score MMA has read the tile, before the value MMA
//    multiplies them by the zero probabilities.
//  * Scores S = Q K^T (M 128, N 64, K 288) and values O += P V (M 128, N 256,
//    K 64): fp32 accumulators in TMEM (four 64-column S / P buffers, O 256
//    columns), P as the TMEM A operand in bf16 (the operand type of V; l sums
//    the fp32 probabilities), the key tile's latent planes as the MN-major B
//    operand.  A score warp and a value warp issue them; eight softmax warps,
//    two a lane quarter, rescale O only when a row's maximum grows by more
//    than 2^8; four epilogue warps store an item while the next one starts.
//  Measured (s = 2, H = 8): 32 single tokens over 2048 rows 20.4 us (1.86 TB/s;
//  seven tiles a block between fixed 13 us), 128 sequences of up to 5 tokens over
//  2048 .. 4096 rows 55.5 us (4.06 TB/s; 62 to 67 at the power cap), four chunks of
//  1024 tokens after 16384 281 to 291 us (1033 to 1070 TFLOP/s).
#include "paged.cuh"

namespace mtla {
namespace ptt {

constexpr int R = 256, DR = 32, D = R + DR;
constexpr int BM = PTC_ROWS;           // rows of an M tile (128)
constexpr int BN = 64;                 // columns of a key tile
constexpr int GRP = D / 32 * 512;      // bytes of an 8-row group: nine planes of 8 x 64 B (4608)
constexpr int QBYTES = BM / 8 * GRP;   // 73728
constexpr int KBYTES = BN / 8 * GRP;   // 36864
constexpr int KS = 5;                  // key-tile stages at most
constexpr int SMW = 8, EPW = 4;        // softmax and epilogue warps
constexpr int TMA_WARP = SMW, SMMA_WARP = SMW + 1, PMMA_WARP = SMW + 2, SCHED_WARP = SMW + 3, EPI_WARP0 = SMW + 4;
constexpr int NT = 32 * (SMW + 4 + EPW);
static_assert(EPI_WARP0 % 4 == 0, "epilogue warp e reads TMEM lane quarter e");
constexpr uint32_t TMEM_COLS = 512, O_COL = 256;
constexpr int NSB = 4;                 // S / P buffers in TMEM (64 columns each)
__host__ __device__ constexpr uint32_t s_col(int b) { return 64u * (uint32_t)b; }
constexpr uint32_t IDESC_O = umma_idesc_bf16(BM, R, false, true);
constexpr int RING = 4;                // items in flight
constexpr int WINS = NT;               // sequence windows kept
constexpr int CONSUMERS = 3 + SMW + EPW;
constexpr int OST_BYTES = 32 * 64;     // output staging of one epilogue warp: 32 rows x 64 bytes

struct RingItem {
  int b, row0, ntok, R;  // ntok == 0: no more items
  int64_t t;
  int kt0, kt1, slot, pad;
};

constexpr size_t OFF_Q = 0;
// Operands: the queries' groups and as many key stages as lie behind those that
// can be live: five behind 40 rows, four behind 64, three behind all 128 (the
// score MMA always reads the place of all 128: what stands in a dead row's
// groups, keys among them, ends in a dead row's scores).
constexpr int Q5_ROWS = 40;
constexpr size_t OPERANDS = Q5_ROWS / 8 * GRP + (size_t)KS * KBYTES;
__host__ __device__ constexpr int stages_of(int rows) { return rows <= Q5_ROWS ? 5 : (rows <= BM / 2 ? 4 : 3); }
__host__ __device__ constexpr uint32_t keys_off(int stages) {
  return stages == 5 ? Q5_ROWS / 8 * GRP : (stages == 4 ? QBYTES / 2 : QBYTES);
}
static_assert(keys_off(4) + 4 * KBYTES <= OPERANDS && keys_off(3) + 3 * KBYTES <= OPERANDS, "stages");
constexpr size_t OFF_OST = OPERANDS;
constexpr size_t OFF_XCH = OFF_OST + (size_t)EPW * OST_BYTES;  // maxima [2][2][BM], sums [2][2][BM], final maxima [2][BM]
constexpr size_t OFF_HID = OFF_XCH + 10 * BM * 4;              // [2] items: a byte a softmax warp that hid values
constexpr size_t OFF_RING = OFF_HID + 2 * SMW;
constexpr size_t OFF_WIN = OFF_RING + RING * sizeof(RingItem);
constexpr size_t OFF_PLAN = OFF_WIN + WINS * sizeof(SeqWin);
constexpr size_t OFF_BAR = (OFF_PLAN + sizeof(PlanShared) + 15) / 16 * 16;
constexpr int NBAR = 2 + 4 + 2 * KS + 3 * NSB + 3 + 2 * RING;
constexpr size_t OFF_TMEM = OFF_BAR + NBAR * 8;
constexpr size_t SMEM = OFF_TMEM + 16 + 1024;
static_assert(OFF_WIN % 16 == 0, "windows hold 64-bit fields");
static_assert(OFF_Q == 0 && GRP % 512 == 0 && KBYTES % 512 == 0 && OFF_OST % 512 == 0, "64-byte swizzle: atoms of 512 bytes");
static_assert(SMEM <= 232448, "one block's shared memory (227 KB)");

// 2^x with the hardware approximation (relative error about 2^-22; 2^-inf = 0)
__device__ __forceinline__ float ex2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16};" ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]),
      "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// mbarrier wait by every lane with a warp-uniform result
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity));
}
// barrier of a pair of softmax warps; true if either passes `fail`
__device__ __forceinline__ bool pair_or(int id, bool fail) {
  uint32_t r;
  asm volatile("{\n .reg .pred f;\n setp.ne.u32 f, %1, 0;\n bar.red.or.pred f, %2, 64, f;\n selp.u32 %0, 1, 0, f;\n}"
               : "=r"(r) : "r"(fail ? 1u : 0u), "r"(id) : "memory");
  return r != 0;
}
// groups of key tile kt that are loaded: cache groups, then the tokens' own
__device__ __forceinline__ int tile_groups(int R8g, int ntok, int kt) {
  const int left = R8g + ((ntok + 7) >> 3) - kt * (BN / 8);
  return left < BN / 8 ? left : BN / 8;
}

// Zeros in the place of the latents of a key tile's columns c0 + c (bit c of
// `hidden`) that are not finite (a warp; see restore_nan).  The score MMA has read
// the tile, the value MMA waits for this warp; another warp may do the same.
static __device__ __noinline__ void hide_latents(uint8_t* stage, int c0, uint32_t hidden) {
  const int lane = threadIdx.x & 31;
  for (; hidden; hidden &= hidden - 1) {
    const int r = c0 + __ffs(hidden) - 1;
    uint4* const at = reinterpret_cast<uint4*>(stage + (r >> 3) * GRP + (lane >> 2) * 512 + (r & 7) * 64 + (lane & 3) * 16);
    const uint4 v = *at;
    *at = make_uint4(finite_or_zero<__nv_bfloat16>(v.x), finite_or_zero<__nv_bfloat16>(v.y),
                     finite_or_zero<__nv_bfloat16>(v.z), finite_or_zero<__nv_bfloat16>(v.w));
  }
  fence_proxy_async_smem();
}
// one of 32 values is not finite: x 0 is NaN then (two a packed instruction)
__device__ __forceinline__ bool not_finite(const float (&x)[32]) {
  uint64_t z[2] = {0, 0}, v;
#pragma unroll
  for (int c = 0; c < 32; c += 2) {
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(x[c]), "f"(x[c + 1]));
    asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(z[c >> 1 & 1]) : "l"(v), "l"(uint64_t(0)));
  }
  float a, b;
  asm("add.rn.f32x2 %0, %0, %1;" : "+l"(z[0]) : "l"(z[1]));
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(z[0]));
  return a + b != 0.f;
}
__device__ __forceinline__ uint32_t low_bits(int n) { return n <= 0 ? 0u : (n >= 32 ? 0xffffffffu : (1u << n) - 1u); }

__global__ void __launch_bounds__(NT, 1) paged_attn_tc_kernel(const __grid_constant__ PagedAttnMaps mp,
                                                              const __grid_constant__ PagedAttnArgs a) {
  extern __shared__ uint8_t smem_raw[];
  // (an offset, not an integer address: the compiler keeps seeing shared memory)
  uint8_t* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint64_t* bar = reinterpret_cast<uint64_t*>(sm + OFF_BAR);
  uint64_t* const q_full = bar;
  uint64_t* const q_empty = bar + 1;            // the item's last score MMA has read Q
  uint64_t* const stat_full = bar + 2;          // [2] an item's row maxima and sums are written
  uint64_t* const stat_empty = bar + 4;         // [2] the epilogue has read them
  uint64_t* const k_full = bar + 6;             // [KS]
  uint64_t* const k_empty = k_full + KS;        // [KS]
  uint64_t* const s_full = k_empty + KS;        // [NSB]
  uint64_t* const p_full = s_full + NSB;        // [NSB]
  uint64_t* const p_empty = p_full + NSB;       // [NSB] the value MMA has read P
  uint64_t* const o_full = p_empty + NSB;
  uint64_t* const o_empty = o_full + 1;
  uint64_t* const mma_done = o_full + 2;
  uint64_t* const it_full = o_full + 3;         // [RING]
  uint64_t* const it_empty = it_full + RING;    // [RING]
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(sm + OFF_TMEM);
  RingItem* ring = reinterpret_cast<RingItem*>(sm + OFF_RING);
  PlanShared* plan = reinterpret_cast<PlanShared*>(sm + OFF_PLAN);
  float* xmax = reinterpret_cast<float*>(sm + OFF_XCH);   // [2 tile parity][2 halves][BM]
  float* xl = xmax + 4 * BM;                              // [2 item parity][2 halves][BM]
  float* xm = xl + 4 * BM;                                // [2 item parity][BM]
  uint8_t* const hid = sm + OFF_HID;                      // [2 item parity][SMW]
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&stat_full[i], SMW);
      mbar_init(&stat_empty[i], EPW);
    }
    for (int i = 0; i < KS; ++i) {
      mbar_init(&k_full[i], 1);
      mbar_init(&k_empty[i], 1);
    }
    for (int i = 0; i < NSB; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], SMW);
      mbar_init(&p_empty[i], 1);
    }
    mbar_init(o_full, 1);
    mbar_init(o_empty, EPW);
    mbar_init(mma_done, 2);
    for (int i = 0; i < RING; ++i) {
      mbar_init(&it_full[i], 1);
      mbar_init(&it_empty[i], CONSUMERS);
    }
    fence_mbar_init();
  }
  if (warp == 0) {
    tmem_alloc(tmem_holder, TMEM_COLS);
    tmem_relinquish();
  }
  if (warp == TMA_WARP && lane == 0) {
    prefetch_tmap(&mp.q);
    prefetch_tmap(&mp.qr);
    prefetch_tmap(&mp.own);
    prefetch_tmap(&mp.cache);
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  SeqWin* const wins = reinterpret_cast<SeqWin*>(sm + OFF_WIN);
  tc_fence_before();
  plan_block<NT, WINS>(a.c, a.p, a.plan, gridDim.x, blockIdx.x, a.dev_err, plan, wins);  // (holds block barriers)
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  const uint32_t sQ = smem_u32(sm + OFF_Q);
  const int H = a.H;
  // key-tile stages: number, and the place of each
  const uint32_t ns = stages_of(plan->most * H), k_off = keys_off(ns);
  auto stage_off = [k_off](uint32_t st) -> uint32_t { return k_off + st * KBYTES; };
  bool ok = true;

  // the next item of the block's share, for one consumer warp
  auto take = [&](uint32_t n, RingItem& it) -> bool {
    const int e = n % RING;
    if (!warp_wait(&it_full[e], (n / RING) & 1)) {
      ok = false;
      return false;
    }
    it = ring[e];
    __syncwarp();
    if (lane == 0) mbar_arrive(&it_empty[e]);
    return it.ntok > 0;
  };

  if (warp == SCHED_WARP) {
    // ======================= scheduler =======================
    ItemWalk walk;
    walk.init(a.c, a.p, a.plan, blockIdx.x, plan, wins);
    SplitDesc desc = {0, 0, 0, 0};
    for (uint32_t n = 0;; ++n) {
      Item item;
      const bool any = walk.next(a.c, a.p, a.plan, &item);
      const int e = n % RING;
      if (n >= (uint32_t)RING && !warp_wait(&it_empty[e], ((n / RING) & 1) ^ 1)) { ok = false; break; }
      if (lane == 0) {
        RingItem r;
        r.b = any ? item.b : 0;
        r.row0 = any ? item.row0 : 0;
        r.ntok = any ? item.ntok : 0;
        r.R = any ? (int)item.R : 0;
        r.t = any ? item.t : 0;
        r.kt0 = any ? item.kt0 : 0;
        r.kt1 = any ? item.kt1 : 0;
        r.slot = any ? item.slot : -1;
        r.pad = 0;
        ring[e] = r;
        mbar_arrive(&it_full[e]);
      }
      __syncwarp();
      if (!any) break;
      if (item.slot >= 0 && item.kt1 == item.kt) {  // a split item ends in this block
        desc.row0 = item.row0;
        desc.ntok = item.ntok;
        desc.first = first_block(a.plan, walk.C, walk.G, walk.item_start);
      }
    }
    if (lane == 0) a.part.desc[blockIdx.x] = desc;
    if (!ok && lane == 0) set_err(a.dev_err, MTLA_DEVERR_TIMEOUT);
  } else if (warp == TMA_WARP) {
    // ======================= TMA producer =======================
    // Lane l of a batch of four key tiles looks up and loads group l: 32 table
    // entries are read at once, one batch ahead.
    const int32_t pool = (int32_t)(a.p.num_pages * a.p.page_rows);
    uint32_t n = 0, kc = 0, st = 0, ph = 0;      // stage of tile kc and its use's parity
    RingItem it;
    for (; take(n, it); ++n) {
      const int R8g = (it.R + 7) >> 3;
      // the page of a group, read ahead of its use (-1: an own group)
      auto look = [&](int g) -> int32_t {
        if (g >= R8g) return -1;
        return __ldg(a.p.table + (int64_t)it.b * a.p.table_pages + div32((uint32_t)(g * 8), a.p.div_rows));
      };
      int32_t cur = 0, nxt = look(it.kt0 * (BN / 8) + lane);
      // queries: the 8-row groups with live rows
      const int live = it.ntok * H, qg = (live + 7) >> 3;
      if (n > 0 && !warp_wait(q_empty, (n - 1) & 1)) { ok = false; break; }
      if (lane == 0) mbar_arrive_expect_tx(q_full, qg * GRP);
      __syncwarp();
      if (lane < qg) {
        tma_load_3d(sm + OFF_Q + lane * GRP, &mp.q, 0, it.row0 * H + 8 * lane, 0, q_full);
        tma_load_2d(sm + OFF_Q + lane * GRP + 8 * 512, &mp.qr, 0, it.row0 * H + 8 * lane, q_full);
      }
      for (int kt = it.kt0; kt < it.kt1 && ok; ++kt, ++kc) {
        const int sub = (kt - it.kt0) & 3;
        if (sub == 0) {
          cur = nxt;
          nxt = kt + 4 < it.kt1 ? look((kt + 4) * (BN / 8) + lane) : 0;
        }
        if (kc >= ns && !warp_wait(&k_empty[st], ph ^ 1)) { ok = false; break; }
        const int ng = tile_groups(R8g, it.ntok, kt);
        if (lane == 0) mbar_arrive_expect_tx(&k_full[st], ng * GRP);
        __syncwarp();
        const int gi = lane - 8 * sub, g = kt * (BN / 8) + gi;  // this lane's group of the tile
        if (gi >= 0 && gi < ng) {
          uint8_t* dst = sm + stage_off(st) + gi * GRP;
          if (g < R8g) {
            // pool row of the group; of a page outside the pool: past its end, where the box fills with zeros
            int32_t row = pool;
            if (cur >= 0 && cur < a.p.num_pages)
              row = cur * a.p.page_rows + (g * 8 - (int)div32((uint32_t)(g * 8), a.p.div_rows) * a.p.page_rows);
            else
              set_err(a.dev_err, MTLA_DEVERR_CAPACITY);
            tma_load_3d(dst, &mp.cache, 0, row, 0, &k_full[st]);
          }
          else tma_load_3d(dst, &mp.own, 0, it.row0 + 8 * (g - R8g), 0, &k_full[st]);
        }
        if (++st == ns) {
          st = 0;
          ph ^= 1;
        }
      }
      if (!ok) break;
    }
    if (!ok && lane == 0) set_err(a.dev_err, MTLA_DEVERR_TIMEOUT);
    // drain: no copy may still be writing shared memory when the block exits
    if (n > 0) warp_wait(q_full, (n - 1) & 1);
    for (uint32_t j = kc > ns ? kc - ns : 0; j < kc; ++j) warp_wait(&k_full[j % ns], (j / ns) & 1);
  } else if (warp == SMMA_WARP || warp == PMMA_WARP) {
    // ======================= MMA issuers =======================
    const bool scores = warp == SMMA_WARP;
    const uint64_t dq0 = umma_desc(sQ, 16, GRP, 4);
    // (the stages' addresses are added to descriptors of the block's base: below 2^18, no carry)
    const uint64_t dk0 = umma_desc(smem_u32(sm), 16, GRP, 4);
    const uint64_t dv0 = umma_desc(smem_u32(sm), 512, GRP, 4);
    uint32_t n = 0, kc = 0, st = 0, ph = 0;
    RingItem it;
    for (; take(n, it) && ok; ++n) {
      const int R8g = (it.R + 7) >> 3;
      if (scores && !warp_wait(q_full, n & 1)) { ok = false; break; }
      for (int kt = it.kt0; kt < it.kt1 && ok; ++kt, ++kc) {
        const int sb = kc % NSB;
        const uint32_t off = stage_off(st);
        // columns in steps of 16 (two groups): a short last tile takes fewer
        const int n16 = (tile_groups(R8g, it.ntok, kt) + 1) >> 1;
        if (scores) {
          // S(j) = Q K(j)^T, once the value MMA of tile j - NSB has read the buffer
          if (!warp_wait(&k_full[st], ph)) { ok = false; break; }
          if (kc >= (uint32_t)NSB && !warp_wait(&p_empty[sb], ((kc / NSB) & 1) ^ 1)) { ok = false; break; }
          tc_fence_after();
          const uint32_t idesc = umma_idesc_bf16(BM, 16, false, false) + ((uint32_t)(n16 - 1) * 2u << 17);
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint64_t ad = dq0 + (uint64_t)(((kk >> 1) * 512 + (kk & 1) * 32) >> 4);
              const uint64_t bd = dk0 + (uint64_t)((off + (kk >> 1) * 512 + (kk & 1) * 32) >> 4);
              umma_bf16(tmem + s_col(sb), ad, bd, idesc, kk > 0 ? 1u : 0u);
            }
            umma_commit(&s_full[sb]);
            if (kt + 1 == it.kt1) umma_commit(q_empty);
          }
        } else {
          // O += P(j) V(j); its completion frees the key stage and the P buffer
          if (!warp_wait(&p_full[sb], (kc / NSB) & 1)) { ok = false; break; }
          if (kt == it.kt0 && n > 0 && !warp_wait(o_empty, (n - 1) & 1)) { ok = false; break; }
          tc_fence_after();
          if (elect_one()) {
            for (int kk = 0; kk < n16; ++kk) {
              const uint64_t bd = dv0 + (uint64_t)((off + kk * 2 * GRP) >> 4);
              umma_bf16_ts(tmem + O_COL, tmem + s_col(sb) + 8 * kk, bd, IDESC_O, (kt > it.kt0 || kk > 0) ? 1u : 0u);
            }
            umma_commit(&k_empty[st]);
            umma_commit(&p_empty[sb]);
            if (kt + 1 == it.kt1) umma_commit(o_full);
          }
        }
        __syncwarp();
        if (++st == ns) {
          st = 0;
          ph ^= 1;
        }
      }
    }
    if (!ok && lane == 0) set_err(a.dev_err, MTLA_DEVERR_TIMEOUT);
    // every MMA of both warps has completed before TMEM is released
    if (elect_one()) umma_commit(mma_done);
    __syncwarp();
    warp_wait(mma_done, 0);
  } else if (warp >= EPI_WARP0) {
    // ======================= epilogue warps =======================
    // warp EPI_WARP0 + e owns rows 32 e .. 32 e + 31 (TMEM lane quarter e): a
    // whole item's rows leave as out = O / l, a part's as O with (m, l).  bf16
    // rows go 64 bytes of 32 rows at a time through a staging block in shared
    // memory (64-byte swizzle), so that a store writes 64 contiguous bytes of 8
    // rows; fp32 rows (parts: few live rows in a decode step, where the chain of
    // 16 such passes took 2 us) go straight from the registers.
    const int qe = warp - EPI_WARP0, i = qe * 32 + lane;
    const uint32_t lane_base = tmem + ((uint32_t)(qe * 32) << 16);
    const uint32_t ost = smem_u32(sm + OFF_OST + (size_t)qe * OST_BYTES);
    const int tr = lane >> 2, tq = lane & 3;
    RingItem it;
    for (uint32_t n = 0; take(n, it); ++n) {
      const int sb2 = n & 1, live = it.ntok * H;
      if (ok && !warp_wait(&stat_full[sb2], (n >> 1) & 1)) ok = false;
      const float m = xm[sb2 * BM + i];
      const float l = xl[(sb2 * 2 + 0) * BM + i] + xl[(sb2 * 2 + 1) * BM + i];
      const bool hidden = *reinterpret_cast<const uint64_t*>(hid + sb2 * SMW) != 0;  // values of columns that some row does not see
      __syncwarp();
      if (lane == 0) mbar_arrive(&stat_empty[sb2]);
      const bool part = it.slot >= 0;
      const int64_t row = part ? (int64_t)it.slot * BM + i : (int64_t)it.row0 * H + i;
      if (i < live) {
        if (part) a.part.ml[row] = make_float2(m, l);
        else if (a.lse) a.lse[row] = (m + log2f(l)) * 0.6931471805599453f;
      }
      const float inv = part ? 1.f : 1.f / l;
      if (ok && !warp_wait(o_full, n & 1)) ok = false;
      tc_fence_after();
      if (qe * 32 >= live) {  // no live row: the warp has nothing of this item
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(o_empty);
        continue;
      }
      if (part || a.out_f32) {                   // fp32: a lane's row, 128 bytes of it at a time
        float* const dst = (part ? a.part.o : static_cast<float*>(a.out)) + row * R;
#pragma unroll 1
        for (int c = 0; c < R / 64; ++c) {
          uint32_t ov[64];
          tmem_ld32(lane_base + O_COL + c * 64, *reinterpret_cast<uint32_t(*)[32]>(&ov[0]));
          tmem_ld32(lane_base + O_COL + c * 64 + 32, *reinterpret_cast<uint32_t(*)[32]>(&ov[32]));
          tmem_wait_ld();
          if (c == R / 64 - 1) {                 // the last read of O: the next item's value MMAs may start
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(o_empty);
          }
          if (i < live) {
#pragma unroll
            for (int e = 0; e < 64; e += 4)
              *reinterpret_cast<float4*>(dst + c * 64 + e) =
                  make_float4(__uint_as_float(ov[e]) * inv, __uint_as_float(ov[e + 1]) * inv,
                              __uint_as_float(ov[e + 2]) * inv, __uint_as_float(ov[e + 3]) * inv);
          }
        }
        if (__builtin_expect(hidden, false))
          restore_nan<__nv_bfloat16>(a, it.b, it.row0, it.t, qe * 32, live < qe * 32 + 32 ? live : qe * 32 + 32,
                                     dst - (int64_t)i * R, true);
        continue;
      }
      __nv_bfloat16* const base = static_cast<__nv_bfloat16*>(a.out) + (row - lane) * R;  // the quarter's first row
#pragma unroll 1
      for (int c = 0; c < R / 32; ++c) {
        uint32_t ov[32], w[16];
        tmem_ld32(lane_base + O_COL + c * 32, ov);
        tmem_wait_ld();
        if (c == R / 32 - 1) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(o_empty);
        }
#pragma unroll
        for (int e = 0; e < 16; ++e)
          w[e] = pack_bf16x2(__uint_as_float(ov[2 * e]) * inv, __uint_as_float(ov[2 * e + 1]) * inv);
        __syncwarp();                            // the previous block's transposed reads are done
#pragma unroll
        for (int q4 = 0; q4 < 4; ++q4) {
          const uint32_t off = (uint32_t)lane * 64u + ((((uint32_t)q4) ^ (((uint32_t)lane >> 1) & 3u)) << 4);
          asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(ost + off), "r"(w[4 * q4]), "r"(w[4 * q4 + 1]),
                       "r"(w[4 * q4 + 2]), "r"(w[4 * q4 + 3]) : "memory");
        }
        __syncwarp();
#pragma unroll
        for (int k8 = 0; k8 < 4; ++k8) {
          const int r = 8 * k8 + tr;             // row of the quarter this lane stores
          if (qe * 32 + r < live) {
            uint32_t v[4];
            const uint32_t off = (uint32_t)r * 64u + ((((uint32_t)tq) ^ (((uint32_t)r >> 1) & 3u)) << 4);
            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                         : "r"(ost + off));
            *reinterpret_cast<uint4*>(base + (int64_t)r * R + c * 32 + tq * 8) = make_uint4(v[0], v[1], v[2], v[3]);
          }
        }
      }
      if (__builtin_expect(hidden, false))
        restore_nan<__nv_bfloat16>(a, it.b, it.row0, it.t, qe * 32, live < qe * 32 + 32 ? live : qe * 32 + 32,
                                   base - (int64_t)qe * 32 * R, false);
    }
    if (!ok && lane == 0) set_err(a.dev_err, MTLA_DEVERR_TIMEOUT);
  } else {
    // ======================= softmax warps =======================
    // warp w: TMEM lane quarter w % 4 and half w / 4 of the tile's 64 columns
    // and of O's 256.  Warps w and w + 4 share rows: they agree on the running
    // maximum every tile (a barrier of the pair; buffers alternate).  A wait
    // that runs out only stops further waiting inside an item, and at an
    // item's start the pair leaves together, so neither waits for the other
    // for good.
    const int qw = warp & 3, hf = warp >> 2, i = qw * 32 + lane;
    const uint32_t lane_base = tmem + ((uint32_t)(qw * 32) << 16);
    const float sl2 = a.scale_log2;
    uint32_t n = 0, kc = 0, st = 0;
    for (;; ++n) {
      RingItem it;
      const bool more = take(n, it);
      if (pair_or(1 + qw, !ok) || !more) break;
      const int live = it.ntok * H, tok = i / H, R8 = (it.R + 7) & ~7;
      const bool on = i < live;
      // columns this row sees: below `seen`, and its own
      // (rows without a token see everything: what they hold is never stored,
      // and they do not keep their warp on the masked path)
      const int seen = on ? rows_below(a.plan, it.t + tok) : 0x7fffffff;
      const int own = on ? R8 + tok : -1;
      float m_run = -INFINITY, l = 0.f;  // l: this half's sum
      bool hides = false;                // this warp has hidden values of the item
      for (int kt = it.kt0; kt < it.kt1; ++kt, ++kc) {
        const int sb = kc % NSB, xb = kc & 1;
        if (ok && !warp_wait(&s_full[sb], (kc / NSB) & 1)) ok = false;
        tc_fence_after();
        if (kt * BN + BN > it.R) {
          // the tile's rows that are neither cache rows nor own states
          const int rows = ((tile_groups(R8 >> 3, it.ntok, kt) + 1) >> 1) * 16;
          for (int r = warp; r < rows; r += SMW) {
            const int v = kt * BN + r;
            if (v >= it.R && (v < R8 || v >= R8 + it.ntok))
              *reinterpret_cast<uint4*>(sm + stage_off(st) + (r >> 3) * GRP + (lane >> 2) * 512 + (r & 7) * 64 +
                                        (lane & 3) * 16) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
        }
        if (qw * 32 < live) {
          uint32_t sr[32];
          tmem_ld32(lane_base + s_col(sb) + 32 * hf, sr);
          tmem_wait_ld();
          float x[32];
#pragma unroll
          for (int c = 0; c < 32; ++c) x[c] = __uint_as_float(sr[c]);
          const int c0 = kt * BN + 32 * hf, nvis = seen - c0;
          if (!__all_sync(0xffffffffu, nvis >= 32)) {  // some row does not see all of these columns
            const int self = own - c0;
            const uint32_t vis = low_bits(nvis) | ((uint32_t)self < 32u ? 1u << self : 0u);
            // columns of the item that this row does not see
            const uint32_t not_mine =
                on ? (low_bits(it.R - c0) | (low_bits(R8 + it.ntok - c0) & ~low_bits(R8 - c0))) & ~vis : 0u;
            if (__any_sync(0xffffffffu, not_mine != 0u) && __builtin_expect(__any_sync(0xffffffffu, not_finite(x)), 0)) {
              // some score is not finite: of a column that its row does not see?
              float z = 0.f;
#pragma unroll
              for (int c = 0; c < 32; ++c)
                if (not_mine >> c & 1) z = fmaf(x[c], 0.f, z);
              if (__any_sync(0xffffffffu, z != 0.f)) {
                hide_latents(sm + stage_off(st), 32 * hf, __reduce_or_sync(0xffffffffu, not_mine));
                hides = true;
              }
            }
#pragma unroll
            for (int c = 0; c < 32; ++c)
              if (!(vis >> c & 1)) x[c] = -INFINITY;
          }
          float mq[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};  // four independent chains
#pragma unroll
          for (int c = 0; c < 32; ++c) mq[c & 3] = fmaxf(mq[c & 3], x[c]);
          // (the scale is positive: the maximum of the scaled scores)
          const float mx = fmaxf(fmaxf(mq[0], mq[1]), fmaxf(mq[2], mq[3])) * sl2;
          // the row's maximum grew by more than 2^8 in either half: agree on it and
          // rescale l and, once the previous value MMA has landed, this half of
          // the row of O (warp-collective); else nothing is exchanged
          tc_fence_before();
          const bool any = pair_or(1 + qw, on && mx > m_run + 8.f);
          tc_fence_after();
          if (any) {
            xmax[(xb * 2 + hf) * BM + i] = mx;
            named_bar(1 + qw, 64);
            const float rmx = fmaxf(mx, xmax[(xb * 2 + (hf ^ 1)) * BM + i]);
            const bool grow = on && rmx > m_run + 8.f;
            const bool resc = grow && m_run != -INFINITY;
            if (kt > it.kt0 && __any_sync(0xffffffffu, resc)) {
              const uint32_t jp = kc - 1;
              if (ok && !warp_wait(&p_empty[jp % NSB], (jp / NSB) & 1)) ok = false;
              tc_fence_after();
              const float f = resc ? exp2f(m_run - rmx) : 1.f;
#pragma unroll 1
              for (int ch = 0; ch < R / 64; ++ch) {
                uint32_t ov[32];
                const uint32_t col = O_COL + 128 * hf + 32 * ch;
                tmem_ld32(lane_base + col, ov);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 32; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * f);
                tmem_st32(lane_base + col, ov);
              }
              tmem_wait_st();
              l *= f;
            }
            if (grow) m_run = rmx;
          }
          const float mref = m_run == -INFINITY ? 0.f : m_run;
          uint32_t pk[16];
          float lq[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int c = 0; c < 32; c += 2) {
            const float p0 = ex2_approx(fmaf(x[c], sl2, -mref)), p1 = ex2_approx(fmaf(x[c + 1], sl2, -mref));
            lq[(c >> 1) & 3] += p0 + p1;
            pk[c >> 1] = pack_bf16x2(p0, p1);
          }
          l += (lq[0] + lq[1]) + (lq[2] + lq[3]);
          tmem_st16(lane_base + s_col(sb) + 16 * hf, pk);
          tmem_wait_st();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[sb]);
        if (++st == ns) st = 0;
      }
      const int sb2 = n & 1;
      if (ok && n >= 2 && !warp_wait(&stat_empty[sb2], ((n >> 1) & 1) ^ 1)) ok = false;
      xl[(sb2 * 2 + hf) * BM + i] = l;
      if (hf == 0) xm[sb2 * BM + i] = m_run;
      if (lane == 0) hid[sb2 * SMW + warp] = hides;
      __syncwarp();
      if (lane == 0) mbar_arrive(&stat_full[sb2]);
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

}  // namespace ptt

cudaError_t launch_paged_attn_tc(const PagedAttnArgs& a, const PagedAttnMaps& m, int grid, cudaStream_t st) {
  static std::atomic<uint64_t> done_mask{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !(done_mask & (1ull << dev))) {
    e = cudaFuncSetAttribute(ptt::paged_attn_tc_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)ptt::SMEM);
    if (e != cudaSuccess) return e;
    if (dev < 64) done_mask |= 1ull << dev;
  }
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(ptt::NT);
  cfg.dynamicSmemBytes = ptt::SMEM;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, ptt::paged_attn_tc_kernel, m, a);
}

}  // namespace mtla
