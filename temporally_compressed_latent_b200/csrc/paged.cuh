// Chunks of new tokens over a paged cache: argument blocks, the token -> sequence
// search, and the work partition of the attention kernels.
#pragma once

#include <atomic>

#include "kernels.cuh"

namespace mtla {

// Division of 32-bit numbers by a divisor the host knows: floor(x / d) =
// floor(x m / 2^64) with m = ceil(2^64 / d) (exact for every 32-bit x and d > 1).
struct FastDiv {
  uint64_t m;  // 0: d == 1
  uint32_t d;
};
inline FastDiv fast_div(uint32_t d) {
  FastDiv f;
  f.d = d;
  f.m = d > 1 ? ~uint64_t(0) / d + 1 : 0;
  return f;
}
__device__ __forceinline__ uint32_t div32(uint32_t x, const FastDiv& f) {
  return f.m ? (uint32_t)__umul64hi((uint64_t)x, f.m) : x;
}

struct ChunkDev {
  int B, N;
  const int32_t* tok_start;  // [B + 1]
  const int32_t* tok_count;  // [B] or null
  const int32_t* t_prev;     // [B]
};
struct PagesDev {
  void* pages;
  int64_t num_pages, row_stride;
  const int32_t* table;      // [B, table_pages]
  int page_rows, table_pages;
  FastDiv div_rows;          // by page_rows
};

// A sequence's part of a chunk: token rows [first, first + n) at times t0 + 1 .. t0 + n.
struct SeqWin {
  int first, n;
  int64_t t0;
};
// Read from the arrays with every value clamped into range, so that no index
// formed from it leaves the token arrays whatever the arrays hold.
__device__ __forceinline__ SeqWin seq_win(const ChunkDev& c, int b) {
  SeqWin w;
  const int s0 = c.tok_start[b], s1 = c.tok_start[b + 1];
  w.first = s0 < 0 ? 0 : (s0 < c.N ? s0 : c.N);
  const int end = s1 < w.first ? w.first : (s1 < c.N ? s1 : c.N);
  w.n = end - w.first;
  if (c.tok_count) {
    const int k = c.tok_count[b];
    if (k < w.n) w.n = k < 0 ? 0 : k;
  }
  w.t0 = c.t_prev[b];
  return w;
}
__device__ __forceinline__ int64_t table_rows(const PagesDev& p) { return (int64_t)p.table_pages * p.page_rows; }

// Pool row of sequence b's cache row g, or -1 (table entry outside the pool).  g < table_rows.
__device__ __forceinline__ int64_t pool_row(const PagesDev& p, int b, int64_t g) {
  const int64_t k = div32((uint32_t)g, p.div_rows);
  const int32_t page = p.table[(int64_t)b * p.table_pages + k];
  return page >= 0 && page < p.num_pages ? (int64_t)page * p.page_rows + (g - k * p.page_rows) : -1;
}

// The sequence that owns token row i: the last b with tok_start[b] <= i, or -1
// (of starts that do not ascend any b, whose window need not hold i: the callers
// look at both of its ends).
// Taken by a whole warp: every round narrows the range 32-fold (two dependent
// loads for 1024 sequences; a binary search by one thread would take ten).
__device__ __forceinline__ int warp_find_seq(const int32_t* tok_start, int B, int i) {
  const int lane = threadIdx.x & 31;
  int lo = -1, hi = B;  // the answer is in [lo, hi)
  while (hi - lo > 1) {
    const int step = (hi - lo - 1 + 31) / 32;
    const int at = lo + 1 + lane * step;
    const bool below = at < hi && tok_start[at] <= i;
    const int c = __popc(__ballot_sync(0xffffffffu, below));  // probes at or below i (a prefix, as tok_start ascends)
    if (c > 0) lo = lo + 1 + (c - 1) * step;
    else hi = lo + 1;
    if (c > 0 && lo + step < hi) hi = lo + step;
    // c == 0: nothing above lo qualifies
  }
  return lo;
}

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

// ----------------------------------------------------------------------------
// RoPE angles: channel pair k turns by pos * base^(-2k/d_R).  The host passes
// the angle of one position as a fraction of a turn in 64-bit fixed point (its
// whole turns drop out), so the product with a position below 2^32 wraps to the
// position's own fraction with an error below 2^-32 of a turn, by two integer
// multiplies; its upper 32 bits give the quarter turn and the rest, whose sine
// and cosine are short polynomials (error below 2^-23).  The angle of position
// 2^31 is as exact as that of position 1.
// ----------------------------------------------------------------------------
constexpr int MAX_ROPE_PAIRS = 288;
struct RopeTable {
  uint64_t turns[MAX_ROPE_PAIRS];
};
__device__ __forceinline__ float2 rope_cos_sin(uint32_t pos, uint64_t turns) {
  const uint32_t f = (uint32_t)((uint64_t)(pos * turns) >> 32);  // fraction of a turn, 2^-32 units
  const uint32_t quarter = (f + (1u << 29)) >> 30;               // nearest quarter turn (mod 4)
  // the rest, |y| <= pi / 4: Taylor polynomials to y^9 and y^8 (next terms
  // below 2e-9 and 3e-8)
  const float y = (float)(int32_t)(f - (quarter << 30)) * 1.4629180792671596e-9f;  // 2 pi 2^-32
  const float z = y * y;
  float sn = fmaf(z, 1.f / 362880.f, -1.f / 5040.f);
  sn = fmaf(z, sn, 1.f / 120.f);
  sn = fmaf(z, sn, -1.f / 6.f);
  sn = fmaf(z * y, sn, y);
  float cn = fmaf(z, 1.f / 40320.f, -1.f / 720.f);
  cn = fmaf(z, cn, 1.f / 24.f);
  cn = fmaf(z, cn, -0.5f);
  cn = fmaf(z, cn, 1.f);
  const float c = quarter & 1 ? sn : cn, s = quarter & 1 ? cn : sn;
  // x = cos, y = sin of the whole angle: signs by quarter
  return make_float2(__uint_as_float(__float_as_uint(c) ^ (((quarter + 1) & 2) << 30)),
                     __uint_as_float(__float_as_uint(s) ^ ((quarter & 2) << 30)));
}

// ----------------------------------------------------------------------------
// Work partition of the paged attention.
//
// An item is (sequence, up to tpt consecutive tokens of its chunk): all their
// heads are the rows of one M tile.  Its columns, in order: the R = ceil(t/s) - 1
// cache rows that its last token sees, padded to a multiple of 8, then the
// tokens' own states (one virtual row a token), cut into key tiles of 8 q rows.
// With kt key tiles an item weighs item_cost + kt.  The weights of all items,
// one after another, form a line of length C that is cut into equal shares,
// one a block: every block streams the same number of key tiles (to one),
// whether the chunk is one token over a long cache (an item spans many
// blocks) or a long prompt (a block takes many items).  Where a cut falls
// inside an item its parts are combined by a second kernel.
//
// kt = ceil((ceil(R/8) + g) / q) with g = ceil(tokens / 8) and R = floor((t - 1)
// / s): nested divisions fold into one,
//   kt = floor((t + 7 s - 1 + 8 s (g + q - 1)) / (8 q s)),
// linear in t, so the sum over a sequence's items is a sum of floors of a
// linear function, which has a closed form (floor_sum).
// ----------------------------------------------------------------------------
struct PlanArgs {
  int s, tpt, q, item_cost;
  int min_share;   // least weight worth a block of its own
  int one_block;   // most weight that one block takes alone
  FastDiv div_s;
};
// sum over i in [0, n) of floor((a i + b) / m), n > 0, 0 < a < m, a small (tpt,
// of at most 16, against m = 8 q s).  With b = m B + c, 0 <= c < m, it is n B and
// the sum of floor((a i + c) / m), whose terms rise from 0 to some K by at most
// one a step: counted by levels, level k (1 <= k <= K) holds the i from
// ceil((m k - c) / a) on, n of them less that.  With m = a M + f and c = a C + d a
// level's ceiling is M k - C + g_k, g_k = ceil((f k - d) / a), and g_(k + a) = g_k +
// f: one walk over a of them gives the sum of all K.  T holds m, b and a n.
template <typename T>
__device__ __forceinline__ int64_t floor_sum_in(T n, T m, T a, T b) {
  const T B = b / m, c = b - B * m, K = (a * (n - 1) + c) / m;
  const T M = m / a, C = c / a, rounds = K / a;
  const int f = (int)(m - M * a), d = (int)(c - C * a), rest = (int)(K - rounds * a);
  int w = -d, g = 0, all = 0, some = 0;  // w = f k - d - a g, in (-a, 0]
  for (int k = 1; k <= (int)a; ++k) {
    w += f;
    if (w > 0) {
      w -= (int)a;
      ++g;
    }
    all += g;
    if (k <= rest) some += g;
  }
  const uint64_t K_ = K, r = rounds;
  const uint64_t ceils = M * (K_ * (K_ + 1) / 2) - C * K_ + (a * f) * (r * (r - 1) / 2) + r * (uint64_t)all +
                         (uint64_t)(rest * f) * r + (uint64_t)some;
  return (int64_t)((uint64_t)n * (B + K_) - ceils);
}
__device__ inline int64_t floor_sum(uint64_t n, uint64_t m, uint32_t a, uint64_t b) {
  // (a 64-bit division takes several times as long as a 32-bit one)
  if ((b + m + a * n) >> 32 == 0) return floor_sum_in<uint32_t>((uint32_t)n, (uint32_t)m, a, (uint32_t)b);
  return floor_sum_in<uint64_t>(n, m, a, b);
}
// cache rows below the query of time t: R = ceil(t / s) - 1 (1 <= t < 2^32)
__device__ __forceinline__ int rows_below(const PlanArgs& a, int64_t t) { return (int)div32((uint32_t)(t - 1), a.div_s); }
// key tiles of an item whose last token has time t and which holds k tokens (q
// is 4 or 8)
__device__ __forceinline__ int item_tiles(const PlanArgs& a, int64_t t, int k) {
  return (((rows_below(a, t) + 7) >> 3) + ((k + 7) >> 3) + a.q - 1) >> (a.q == 8 ? 3 : 2);
}
// weight of a sequence's first m items (chunk of n tokens after t0).  (Of a
// sequence with several: out of line, a kernel's start over single tokens
// should not have to fetch past this code.)  A few are added one by one; the
// closed form's 64-bit divisions take as long as some dozens.
constexpr int ADD_ITEMS = 32;
static __device__ __noinline__ int64_t items_weight_many(int s, int tpt, int q, int item_cost, FastDiv div_s, int64_t t0, int n,
                                                         int64_t m) {
  const PlanArgs a = {s, tpt, q, item_cost, 0, 0, div_s};
  int64_t w = m * a.item_cost;
  if (m <= ADD_ITEMS) {
    for (int i = 0; i < (int)m; ++i) {
      const int e = (i + 1) * a.tpt < n ? (i + 1) * a.tpt : n;  // tokens up to the item's end
      w += item_tiles(a, t0 + e, e - i * a.tpt);
    }
    return w;
  }
  const int64_t full = n / a.tpt, k = m < full ? m : full;
  w += floor_sum((uint64_t)k, 8ull * a.q * a.s, (uint32_t)a.tpt,
                 (uint64_t)(t0 + a.tpt + 7ll * a.s - 1 + 8ll * a.s * (((a.tpt + 7) >> 3) + a.q - 1)));
  if (m > full) w += item_tiles(a, t0 + n, n - (int)full * a.tpt);
  return w;
}
__device__ __forceinline__ int64_t items_weight(const PlanArgs& a, int64_t t0, int n, int64_t m) {
  if (m == 0) return 0;
  if (n <= a.tpt) return a.item_cost + item_tiles(a, t0 + n, n);  // one item
  return items_weight_many(a.s, a.tpt, a.q, a.item_cost, a.div_s, t0, n, m);
}
// weight of all of a sequence's items
__device__ __forceinline__ int64_t seq_weight(const PlanArgs& a, int64_t t0, int n) {
  if (n <= a.tpt) return n > 0 ? a.item_cost + item_tiles(a, t0 + n, n) : 0;
  return items_weight_many(a.s, a.tpt, a.q, a.item_cost, a.div_s, t0, n, (n + a.tpt - 1) / a.tpt);
}
// The item of a sequence with several that holds offset rem of its weight: the
// largest whose earlier items weigh no more (32 candidates a round, by a warp).
static __device__ __noinline__ int find_item(int s, int tpt, int q, int item_cost, FastDiv div_s, int64_t t0, int n, int64_t rem) {
  const int lane = threadIdx.x & 31;
  int lo = 0, up = (n + tpt - 1) / tpt;
  while (up - lo > 1) {
    const int step = (up - lo - 1 + 31) / 32, at = lo + 1 + lane * step;
    const bool le = at < up && items_weight_many(s, tpt, q, item_cost, div_s, t0, n, at) <= rem;
    const int k = __popc(__ballot_sync(0xffffffffu, le));
    if (k == 0) {
      up = lo + 1;
    } else {
      lo = lo + 1 + (k - 1) * step;
      if (lo + step < up) up = lo + step;
    }
  }
  return lo;
}

// One item's part in a block.
struct Item {
  int b;            // sequence
  int row0, ntok;   // token rows [row0, row0 + ntok)
  int64_t t;        // time of the first of them
  int64_t R;        // cache rows its last token sees
  int kt0, kt1;     // key tiles of this part
  int kt;           // key tiles of the item
  int slot;         // partial-result slot, or -1: the whole item is here, its results go out directly
};

// An upper bound of the blocks that get a share, from what the host knows (N
// tokens of B sequences, tables of `rows` cache rows).  Where it is one, no item
// is split and nothing is left to join.
inline int64_t most_tiles(const PlanArgs& a, int64_t N, int64_t rows) {  // of an item
  return ((rows + 7) / 8 + ((a.tpt < N ? a.tpt : N) + 7) / 8 + a.q - 1) / a.q;
}
inline int most_blocks(const PlanArgs& a, int64_t N, int64_t B, int64_t rows, int grid) {
  int64_t items = (N + a.tpt - 1) / a.tpt + B;
  if (items > N) items = N;
  const int64_t C = items * (a.item_cost + most_tiles(a, N, rows));
  if (C <= a.one_block) return 1;
  const int64_t g = (C + a.min_share - 1) / a.min_share;
  return g < grid ? (int)g : grid;
}
// Blocks that get a share: no more than give each min_share of the weight C.
__device__ __forceinline__ int64_t share_blocks(const PlanArgs& a, int64_t C, int grid) {
  if (C >= (int64_t)a.min_share * grid) return grid;
  if (C <= a.one_block) return C > 0;  // too little to pay for joining parts
  return ((int)C + a.min_share - 1) / a.min_share;
}
// Shares: block x of G takes [C x / G, C (x + 1) / G).
__device__ __forceinline__ int64_t share_lo(int64_t C, int64_t G, int64_t x) {
  // (a 64-bit division is a few hundred cycles of one warp's time)
  if (C < (1 << 20)) return (uint32_t)C * (uint32_t)x / (uint32_t)G;  // G < 2^12
  return C * x / G;
}

struct PlanShared {
  int64_t warp_sum[32];
  int64_t C, G, before;  // total weight; blocks with a share; weight of the sequences before `b`
  int b;                 // sequence holding this block's first position
  int kept;              // windows in win
  int most;              // most tokens of an item
};

// The chunk window the attention takes (a sequence whose rows exceed its table,
// or whose times leave [0, 2^31), takes none: those that the append refuses for
// want of room have no states to attend).
__device__ __forceinline__ SeqWin attn_win(const ChunkDev& c, const PagesDev& p, const FastDiv& div_s, int b,
                                           int32_t* dev_err) {
  SeqWin w = seq_win(c, b);
  if (w.n > 0 && (w.t0 < 0 || w.t0 + w.n > 0x7fffffff || (int64_t)div32((uint32_t)(w.t0 + w.n - 1), div_s) >= table_rows(p))) {
    if (dev_err) set_err(dev_err, MTLA_DEVERR_CAPACITY);
    w.n = 0;
  }
  return w;
}

// Taken by every thread of the block: the total weight C, and the sequence
// that holds position share_lo(C, G, x).  One pass over the sequences (each
// thread sums a run of them) and one block scan; the thread whose run holds
// the position walks its run again.  win: of no more than WINS <= NT sequences
// the windows are kept here for the walk.
template <int NT, int WINS>
__device__ inline void plan_block(const ChunkDev& c, const PagesDev& p, const PlanArgs& a, int grid, int x,
                                  int32_t* dev_err, PlanShared* sh, SeqWin* win) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (c.B + NT - 1) / NT;
  const int b0 = tid * per < c.B ? tid * per : c.B, b1 = b0 + per < c.B ? b0 + per : c.B;
  int64_t sum = 0;
  int most = 0;
  if (tid == 0) sh->most = 0;
  for (int b = b0; b < b1; ++b) {
    const SeqWin w = attn_win(c, p, a.div_s, b, x == 0 ? dev_err : nullptr);
    sum += seq_weight(a, w.t0, w.n);
    most = most > w.n ? most : w.n;
    if (c.B <= WINS) win[b] = w;
  }
  most = (int)__reduce_max_sync(0xffffffffu, (unsigned)(most < a.tpt ? most : a.tpt));
  int64_t pre = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xffffffffu, pre, o);
    if (lane >= o) pre += v;
  }
  if (lane == 31) sh->warp_sum[warp] = pre;
  if (tid == 0) sh->b = -1;
  __syncthreads();
  if (lane == 0) atomicMax(&sh->most, most);
  int64_t base = 0, C = 0;
  const int warps = per == 1 ? (c.B + 31) / 32 : NT / 32;  // warps that have sequences
  for (int w = 0; w < warps; ++w) {
    if (w < warp) base += sh->warp_sum[w];
    C += sh->warp_sum[w];
  }
  const int64_t G = share_blocks(a, C, grid);
  if (tid == 0) {
    sh->C = C;
    sh->G = G;
    sh->kept = c.B <= WINS;
  }
  if (x < G) {
    const int64_t lo = share_lo(C, G, x);
    int64_t at = base + pre - sum;
    if (lo >= at && lo < at + sum) {
      int b = b0;
      for (; b + 1 < b1; ++b) {  // (not taken where every thread has one)
        const SeqWin w = attn_win(c, p, a.div_s, b, nullptr);
        const int64_t k = seq_weight(a, w.t0, w.n);
        if (lo < at + k) break;
        at += k;
      }
      sh->b = b;
      sh->before = at;
    }
  }
  __syncthreads();
}

// Walks the items of block x's share in order.  Every lane of one warp calls
// init and next together; results are warp-uniform.
struct ItemWalk {
  int64_t pos, hi, C, G;
  int64_t start;          // position of the current item
  int b, tile, x;
  int batch;              // first sequence of the window batch in the lanes
  int w_first, w_n;       // this lane's sequence batch + lane
  int64_t w_t0;
  const SeqWin* win;      // the plan's windows, or null

  __device__ __forceinline__ void load(const ChunkDev& c, const PagesDev& p, const PlanArgs& a, int b0) {
    batch = b0;
    const int bb = b0 + (threadIdx.x & 31);
    SeqWin w;
    w.first = 0;
    w.n = 0;
    w.t0 = 0;
    if (bb < c.B) w = win ? win[bb] : attn_win(c, p, a.div_s, bb, nullptr);
    w_first = w.first;
    w_n = w.n;
    w_t0 = w.t0;
  }

  __device__ inline void init(const ChunkDev& c, const PagesDev& p, const PlanArgs& a, int x_, const PlanShared* sh,
                              const SeqWin* wins) {
    x = x_;
    C = sh->C;
    G = sh->G;
    win = sh->kept ? wins : nullptr;
    if (x >= G || sh->b < 0) {
      pos = hi = 0;
      return;
    }
    pos = share_lo(C, G, x);
    hi = share_lo(C, G, x + 1);
    b = sh->b;
    load(c, p, a, b);
    const int n = __shfl_sync(0xffffffffu, w_n, 0);
    const int64_t t0 = __shfl_sync(0xffffffffu, w_t0, 0);
    tile = n <= a.tpt ? 0 : find_item(a.s, a.tpt, a.q, a.item_cost, a.div_s, t0, n, pos - sh->before);
    start = sh->before + items_weight(a, t0, n, tile);
  }

  // The next item with key tiles in this share; false at the share's end.
  __device__ inline bool next(const ChunkDev& c, const PagesDev& p, const PlanArgs& a, Item* it) {
    while (pos < hi) {
      const int src = b - batch;
      const int first = __shfl_sync(0xffffffffu, w_first, src), n = __shfl_sync(0xffffffffu, w_n, src);
      const int64_t t0 = __shfl_sync(0xffffffffu, w_t0, src);
      const int i0 = tile * a.tpt, k = n - i0 < a.tpt ? n - i0 : a.tpt;
      const int kt = item_tiles(a, t0 + i0 + k, k);
      const int64_t end = start + a.item_cost + kt;
      const int64_t y = hi < end ? hi : end;
      const int64_t k0 = pos - start - a.item_cost, k1 = y - start - a.item_cost;
      it->b = b;
      it->row0 = first + i0;
      it->ntok = k;
      it->t = t0 + i0 + 1;
      it->R = rows_below(a, t0 + i0 + k);
      it->kt0 = k0 > 0 ? (int)k0 : 0;
      it->kt1 = k1 > 0 ? (int)k1 : 0;
      it->kt = kt;
      // outgoing parts (the item starts here and goes on) use slot 2 x + 1,
      // the others 2 x: a block has at most one of each
      it->slot = it->kt0 == 0 && it->kt1 == it->kt ? -1 : (it->kt0 == 0 ? 2 * x + 1 : 2 * x);
      const bool some = it->kt1 > it->kt0;
      item_start = start;
      pos = y;
      if (y == end) {  // on to the next item
        start = end;
        ++tile;
        if (tile * a.tpt >= n) {
          tile = 0;
          ++b;
          while (pos < hi) {  // the next sequence with tokens (one exists: positions are left)
            if (b - batch >= 32) load(c, p, a, b);
            const uint32_t has = __ballot_sync(0xffffffffu, w_n > 0) & (0xffffffffu << (b - batch));
            if (has) {
              b = batch + __ffs(has) - 1;
              break;
            }
            b = batch + 32;
            if (b >= c.B) {
              pos = hi;
              break;
            }
          }
        }
      }
      if (some) return true;
    }
    return false;
  }
  int64_t item_start;     // position of the item that next() returned
};

// What a block tells the combine kernel: the split item that ends in it.
struct SplitDesc {
  int row0, ntok;   // ntok == 0: none
  int first;        // first block with a part of it
  int pad;
};
// The first block that holds a key tile of an item at position `start`: the
// last x with share_lo(x) <= start + item_cost.
__device__ __forceinline__ int first_block(const PlanArgs& a, int64_t C, int64_t G, int64_t start) {
  if (C < (1 << 20)) return (int)(((uint32_t)(start + a.item_cost + 1) * (uint32_t)G - 1u) / (uint32_t)C);
  return (int)(((start + a.item_cost + 1) * G - 1) / C);
}

// Partial results: slot (2 a block), row of the M tile: (max, sum) in log2
// units and the unnormalised output, fp32.
struct PartBuf {
  SplitDesc* desc;  // [grid]
  float2* ml;       // [2 grid][rows]
  float* o;         // [2 grid][rows][r]
};
struct PagedLayout {
  size_t desc, ml, o, total;
};
inline PagedLayout paged_layout(int grid, int rows, int r) {
  auto up = [](size_t x) { return (x + 255) & ~(size_t)255; };
  PagedLayout l;
  l.desc = 0;
  l.ml = up((size_t)grid * sizeof(SplitDesc));
  l.o = l.ml + up((size_t)2 * grid * rows * 8);
  l.total = l.o + up((size_t)2 * grid * rows * r * 4);
  return l;
}

struct PagedAttnArgs {
  ChunkDev c;
  PagesDev p;
  PlanArgs plan;
  PartBuf part;
  const void *q_abs, *q_rope, *row_state;
  void* out;
  float* lse;
  int32_t* dev_err;
  int H, r, d_R;
  int out_f32;
  int rows;          // rows of an M tile (stride of the partial buffers)
  float scale_log2;  // log2(e) / sqrt(d_h)
};

// ----------------------------------------------------------------------------
// NaN and infinite values of an item's keys.
//
// The rows of an M tile share every key tile, so the value product also takes
// columns that some of its rows do not see (a later token's own state, a group
// that a later token closed), with probability zero; 0 x NaN and 0 x inf would
// hand a later token's values to an earlier one.  Such a column's score is itself
// not finite, whatever the query.  So where a hidden score is not finite, the
// column's latents that are not finite become zeros before the value product,
// and the rows that do see the column get their NaN back when the item is stored
// (p v is NaN for every such v that a row sees: its score is NaN or +inf, and with
// it every p, or -inf, and p = 0).  Ordinary values pay for the look alone.
// ----------------------------------------------------------------------------
// the elements of a 32-bit word that are not finite, as zeros
template <typename T> __device__ __forceinline__ uint32_t finite_or_zero(uint32_t w);
template <> __device__ __forceinline__ uint32_t finite_or_zero<float>(uint32_t w) { return (w & 0x7f800000u) == 0x7f800000u ? 0u : w; }
template <> __device__ __forceinline__ uint32_t finite_or_zero<__nv_bfloat16>(uint32_t w) {
  if ((w & 0x7f80u) == 0x7f80u) w &= 0xffff0000u;
  return (w & 0x7f800000u) == 0x7f800000u ? w & 0xffffu : w;
}
// Rows [i0, i1) of an item's M tile (a multiple of r elements apart from dst, row
// 0's; fp32 or T), by the warp that has stored them: NaN in every channel in which
// a column that the row sees, and that not all rows of the item see, is not finite.
template <typename T>
static __device__ __noinline__ void restore_nan(const PagedAttnArgs& a, int b, int row0, int64_t t, int i0, int i1, void* dst,
                                                bool f32) {
  const int lane = threadIdx.x & 31;
  const int64_t g0 = rows_below(a.plan, t);
  __syncwarp();
  for (int i = i0; i < i1; ++i) {
    const int tok = i / a.H;
    const int64_t g1 = rows_below(a.plan, t + tok);
    for (int64_t g = g0; g <= g1; ++g) {
      const T* src = reinterpret_cast<const T*>(a.row_state) + (int64_t)(row0 + tok) * (a.r + a.d_R);
      if (g < g1) {
        const int64_t row = pool_row(a.p, b, g);
        if (row < 0) continue;
        src = reinterpret_cast<const T*>(a.p.pages) + row * a.p.row_stride;
      }
      for (int e = lane; e < a.r; e += 32) {
        if (isfinite(ld_f32(src + e))) continue;
        const int64_t at = (int64_t)i * a.r + e;
        if (f32) reinterpret_cast<float*>(dst)[at] = __int_as_float(0x7fc00000);
        else st_elem(reinterpret_cast<T*>(dst) + at, __int_as_float(0x7fc00000));
      }
    }
  }
}

// generic kernel (paged_attn.cu)
constexpr int PSM = 32;  // M tile rows
constexpr int PSN = 32;  // key tile rows
int paged_simt_grid(int r, int d_R, int dtype, int sms);  // blocks of its persistent grid (0 on error)
cudaError_t launch_paged_attn_simt(const PagedAttnArgs& a, int grid, int dtype, cudaStream_t st);
cudaError_t launch_paged_combine(const PagedAttnArgs& a, int grid, int sms, int dtype, cudaStream_t st);

// tensor-core kernel (paged_attn_tc.cu): bf16, r = 256, d_R = 32
constexpr int PTC_ROWS = 128;  // M tile rows
constexpr int PTC_COLS = 64;   // key tile columns
struct PagedAttnMaps {
  CUtensorMap q;      // q_abs as {32, N H rows, 8 planes}, boxes of 8 rows
  CUtensorMap qr;     // q_rope {32, N H rows}, boxes of 8 rows
  CUtensorMap own;    // row_state {32, N, 9 planes}, boxes of 8 rows
  CUtensorMap cache;  // pages {32, pool rows, 9 planes}, boxes of 8 rows
};
cudaError_t launch_paged_attn_tc(const PagedAttnArgs& a, const PagedAttnMaps& m, int grid, cudaStream_t st);

struct PagedAppendArgs {
  ChunkDev c;
  PagesDev p;
  MergeArgsDev m;
  RopeTable rope;
  const void* q_rope;
  void* q_rope_out;
  const float* tail_in;
  float* tail_out;
  int32_t *t_out, *cache_len;
  void* row_state;
  int32_t* dev_err;
  int H, r, d_R, s;
  FastDiv div_s;
  int rotate;  // 0: keys and queries are rotated already
  int tt;      // tokens of a block's tile (generic kernel)
  int halo;    // token rows before a tile that its block always computes too, or -1: as many as its first group needs
};
// The chunk window the append takes: a sequence that does not fit its table or
// the P table (or whose times leave [0, 2^31)) takes none.  Divisions by s are
// 32-bit.
using AppendWin = SeqWin;
__device__ __forceinline__ void append_fit(const PagedAppendArgs& a, AppendWin& w, bool report) {
  if (w.n > 0) {
    const uint32_t j = div32((uint32_t)w.t0 + (uint32_t)w.n - 1u, a.div_s) + 1u;  // (of a t0 >= 0)
    const bool cap = w.t0 < 0 || w.t0 + w.n > 0x7fffffff || j > table_rows(a.p), pe = !cap && j > (uint32_t)a.m.J_max;
    if (cap || pe) {
      if (report) set_err(a.dev_err, cap ? MTLA_DEVERR_CAPACITY : MTLA_DEVERR_PE_RANGE);
      w.n = 0;
    }
  }
}
__device__ __forceinline__ AppendWin append_win(const PagedAppendArgs& a, int b, bool report) {
  SeqWin w = seq_win(a.c, b);
  append_fit(a, w, report);
  return w;
}
// The sequence (-1: none) and append window of token row base + lane, by a whole
// warp: one round of loads for up to 32 sequences (a lane each), else a search
// and a second round.
__device__ __forceinline__ void warp_windows(const PagedAppendArgs& a, int64_t base, int& b, AppendWin& w) {
  const int lane = threadIdx.x & 31;
  if (a.c.B <= 32) {
    AppendWin mine;
    mine.first = mine.n = 0;
    mine.t0 = 0;
    int start = 0x7fffffff;
    if (lane < a.c.B) {
      start = a.c.tok_start[lane];
      mine = append_win(a, lane, false);
    }
    b = -1;
    for (int k = 0; k < a.c.B; ++k)
      if (__shfl_sync(0xffffffffu, start, k) <= base + lane) b = k;
    const int from = b < 0 ? 0 : b;
    w.first = __shfl_sync(0xffffffffu, mine.first, from);
    w.n = __shfl_sync(0xffffffffu, mine.n, from);
    w.t0 = __shfl_sync(0xffffffffu, mine.t0, from);
  } else {
    int v[1];
    warp_sequences<1>(a.c, base, v);
    b = v[0];
    w = append_win(a, b < 0 ? 0 : b, false);
  }
}
cudaError_t launch_paged_append_simt(PagedAppendArgs& a, int dtype, int sms, cudaStream_t st);

// tensor-core kernel (paged_append_tc.cu): bf16, r = 256, d_R = 32, s <= 64
constexpr int PTA_MAX_S = 64;
struct PagedAppendMaps {
  CUtensorMap c;   // c_new {256, N}, boxes of 64 x 128 rows, 128-byte swizzle
  CUtensorMap kr;  // kR_new {32, N}, boxes of 128 rows
};
cudaError_t launch_paged_append_tc(const PagedAppendArgs& a, const PagedAppendMaps& m, int sms, cudaStream_t st);

struct VerifyArgs {
  int B, N, V;
  const float *p, *q;
  int64_t ld_p, ld_q;
  const int32_t *tokens, *tok_start;
  const float *u_accept, *u_sample;
  int32_t *n_keep, *next_token;
  int32_t* dev_err;
};
cudaError_t launch_verify(const VerifyArgs& a, int sms, cudaStream_t st);

}  // namespace mtla
