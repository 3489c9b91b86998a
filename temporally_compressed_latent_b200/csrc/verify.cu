// Verification of drafted tokens against the target's probabilities, from given
// random numbers (speculative sampling).
//
// Draft x, drawn from q, is kept with probability min(1, p(x) / q(x)): iff
// u q(x) < p(x).  At the first draft dropped, the next token comes from the
// residual max(p - q, 0), so that kept and drawn tokens together follow p; when
// all are kept, from p of the chunk's last row.  It is drawn by inversion: the
// lowest index whose running sum exceeds u times the sum.
//
// A cluster of up to 16 blocks takes a sequence: only one row of p and of q is
// read (the drafts' probabilities are gathers), so the vocabulary is split over
// the cluster for its latency and bandwidth, and the blocks exchange their sums
// through distributed shared memory.  A warp sums 256 entries at a time, eight
// a lane, and notes each sum; after the exchange the one block that holds the
// drawn index scans its sums and reads one such run again.  Runs are cut at
// 16-byte boundaries of p's row, so rows of any alignment are read four entries
// a load.  Sums are in double precision: the running sum over 10^5 entries of
// size 10^-5 must place the border between neighbours, which 24 bits would miss
// once in a hundred draws.  They are trees of depth three in a lane and five
// across it (an addition in double takes tens of cycles: chains of 32 made one
// sequence's call 17 us instead of 5).
// Bound by the two rows' HBM reads (large batches: 96 rows of 131072 take 20.6 us,
// 4.8 TB/s) or by the chain of four dependent reads and the cluster's barriers
// (small ones: one row of 32000 5.2 us).
#include <cooperative_groups.h>

#include "paged.cuh"

namespace mtla {
namespace vfy {

namespace cg = cooperative_groups;
constexpr int MAXCL = 16;
constexpr int NT = 256, NW = NT / 32, BLOCKS = 3;   // threads; resident blocks an SM (of 4, 64 registers spill: 96 x 131072 2.5 us longer)
constexpr int RUN = 256;                            // entries a warp sums at a time
constexpr int MAXRUNS = 4104;                       // runs of a block (2^22 entries over 4 blocks: 4097)

// entries that are NaN, infinite or not above zero count as zero
__device__ __forceinline__ float clean(float x) { return x > 0.f && x <= 3.4028234663852886e38f ? x : 0.f; }
__device__ __forceinline__ double warp_sum(double x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}
__device__ __forceinline__ double warp_scan(double x) {  // inclusive
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const double y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x;
}

// What the next token is drawn from.  Entries are counted from the 16-byte
// boundary at or before the row's start: position j is entry j - shift.
struct Weights {
  const float *p, *q;   // q: null where p alone counts
  int V, hole;          // hole: an entry without weight, or -1
  int shift;            // entries between that boundary and the row of p
  bool qvec;            // q is absent or its row has the same shift
  // eight positions of a run starting at j0: lane l's are j0 + 4 l .. + 3 and
  // j0 + 128 + 4 l .. + 3; those outside the row, and all of an absent q, are zero
  __device__ __forceinline__ void load(int j0, float (&a)[8], float (&b)[8]) const {
    const int v0 = j0 + 4 * (threadIdx.x & 31) - shift;
    if (j0 >= shift && j0 + RUN - shift <= V && qvec) {  // (warp-uniform) the whole run, in quadruples
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float4 x = __ldg(reinterpret_cast<const float4*>(p + v0 + 128 * h));
        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
        if (q) y = __ldg(reinterpret_cast<const float4*>(q + v0 + 128 * h));
        a[4 * h] = x.x; a[4 * h + 1] = x.y; a[4 * h + 2] = x.z; a[4 * h + 3] = x.w;
        b[4 * h] = y.x; b[4 * h + 1] = y.y; b[4 * h + 2] = y.z; b[4 * h + 3] = y.w;
      }
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int v = v0 + 128 * (k >> 2) + (k & 3);
        const bool in = v >= 0 && v < V;
        a[k] = in ? __ldg(p + v) : 0.f;
        b[k] = in && q ? __ldg(q + v) : 0.f;
      }
    }
  }
  __device__ __forceinline__ void weigh(int j0, float (&a)[8], float (&b)[8], double (&w)[8]) const {
    // one comparison for all of a lane's entries: as unsigned, the bits of those
    // that do not count are the largest
    uint32_t top = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) top = max(max(top, __float_as_uint(a[k])), __float_as_uint(b[k]));
    if (top >= 0x7f800000u) {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        a[k] = clean(a[k]);
        b[k] = clean(b[k]);
      }
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) w[k] = (double)fmaxf(a[k], b[k]) - (double)b[k];
    const int at = hole + shift - j0;  // the hole's position in this run
    if (hole >= 0 && at >= 0 && at < RUN) {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (128 * (k >> 2) + 4 * (int)(threadIdx.x & 31) + (k & 3) == at) w[k] = 0.0;
    }
  }
  // the sum of a run's weights, to every lane
  __device__ __forceinline__ double sum(int j0, float (&a)[8], float (&b)[8]) const {
    double x[8];
    weigh(j0, a, b, x);
    return warp_sum(((x[0] + x[1]) + (x[2] + x[3])) + ((x[4] + x[5]) + (x[6] + x[7])));
  }
};

__global__ void __launch_bounds__(NT, BLOCKS) verify_kernel(const VerifyArgs a) {
  cg::cluster_group cluster = cg::this_cluster();
  __shared__ double run_sum[MAXRUNS];
  __shared__ double warp_total[NW];
  __shared__ double totals[2][MAXCL];                 // every block's sum, written by the blocks themselves
  __shared__ int first_drop;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int CL = (int)cluster.num_blocks(), rank = (int)cluster.block_rank(), b = blockIdx.x / CL;

  const int s0 = a.tok_start[b], s1 = a.tok_start[b + 1];
  const int first = s0 < 0 ? 0 : (s0 < a.N ? s0 : a.N);
  const int end = s1 < first ? first : (s1 < a.N ? s1 : a.N), n = end - first;
  if (n == 0) {  // the whole cluster leaves
    if (rank == 0 && tid == 0) {
      a.n_keep[b] = 0;
      a.next_token[b] = -1;
    }
    return;
  }
  // (the blocks of the cluster have all started when the first sum is sent)
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  const float u = a.u_sample[b];
  // ---- the first draft dropped (n - 1: none); every block finds it for itself
  if (tid == 0) first_drop = n - 1;
  __syncthreads();
  for (int i0 = 0; i0 < n - 1; i0 += NT) {
    const int i = i0 + tid;
    if (i < n - 1) {
      const int64_t row = first + i;
      const int x = a.tokens[row + 1];
      const float ua = a.u_accept[row];
      bool keep = false;
      if (x >= 0 && x < a.V) {
        const double p = clean(a.p[row * a.ld_p + x]), q = a.q ? clean(a.q[row * a.ld_q + x]) : 1.f;
        keep = (double)ua * q < p;
      } else if (rank == 0) {
        set_err(a.dev_err, MTLA_DEVERR_TOKEN);
      }
      if (!keep) atomicMin(&first_drop, i);
    }
    __syncthreads();
    if (first_drop < i0 + NT) break;
  }
  const int drop = first_drop;
  const bool dropped = drop < n - 1;
  Weights w;
  w.p = a.p + (int64_t)(first + drop) * a.ld_p;
  w.q = a.q && dropped ? a.q + (int64_t)(first + drop) * a.ld_q : nullptr;
  w.V = a.V;
  w.shift = (int)(reinterpret_cast<uintptr_t>(w.p) >> 2 & 3);
  w.qvec = !w.q || (int)(reinterpret_cast<uintptr_t>(w.q) >> 2 & 3) == w.shift;
  // certain drafts (no q): the residual is p without the dropped token
  w.hole = !a.q && dropped ? a.tokens[first + drop + 1] : -1;

  const int runs = (a.V + w.shift + RUN - 1) / RUN, per = (runs + CL - 1) / CL;
  const int r_beg = rank * per < runs ? rank * per : runs, r_end = r_beg + per < runs ? r_beg + per : runs;
  const int mine = r_end - r_beg;
  double total = 0.0;
  int round = 0;
  for (;; ++round) {
    double sum = 0.0;
    // the next run's loads are in flight while one is summed
    float pa[8], qa[8], pb[8], qb[8];
    if (warp < mine) w.load((r_beg + warp) * RUN, pa, qa);
    for (int r = warp; r < mine; r += 2 * NW) {
      const bool more = r + NW < mine;
      if (more) w.load((r_beg + r + NW) * RUN, pb, qb);
      double s = w.sum((r_beg + r) * RUN, pa, qa);
      if (lane == 0) run_sum[r] = s;
      sum += s;
      if (!more) break;
      if (r + 2 * NW < mine) w.load((r_beg + r + 2 * NW) * RUN, pa, qa);
      s = w.sum((r_beg + r + NW) * RUN, pb, qb);
      if (lane == 0) run_sum[r + NW] = s;
      sum += s;
    }
    if (lane == 0) warp_total[warp] = sum;
    if (round == 0) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    __syncthreads();
    if (warp == 0) {
      const double s = warp_sum(lane < NW ? warp_total[lane] : 0.0);
      // to every block of the cluster (two buffers: a second round's sums do
      // not meet late readers of the first's)
      if (lane < CL) *cluster.map_shared_rank(&totals[round & 1][rank], lane) = s;
    }
    cluster.sync();
    total = 0.0;
    for (int r = 0; r < CL; ++r) total += totals[round & 1][r];
    if (total > 0.0 || !dropped || round > 0) break;
    w.q = nullptr;  // nothing above q: draw from p
    w.qvec = true;
    w.hole = -1;
  }
  if (rank == 0 && tid == 0) a.n_keep[b] = drop + 1;
  if (!(total > 0.0)) {
    if (rank == 0 && tid == 0) {
      a.next_token[b] = -1;
      set_err(a.dev_err, MTLA_DEVERR_EMPTY);
    }
    return;
  }
  // ---- the block, the run and the entry where the running sum passes the target
  const double target = (u > 0.f ? (double)u : 0.0) * total;
  int owner = -1;
  double before = 0.0;
  {
    double c = 0.0;
    for (int r = 0; r < CL; ++r) {
      const double t = totals[round & 1][r];
      if (t > 0.0) {
        // (the last block with any weight takes what rounding leaves over)
        owner = r;
        before = c;
        if (c + t > target) break;
      }
      c += t;
    }
  }
  if (owner != rank || warp != 0) return;
  // warp 0 scans the sums of the block's runs, 32 at a time; the last run with
  // any weight takes what rounding leaves over
  int pick = -1;
  double at = before, c = before;
  for (int r0 = 0; r0 < mine; r0 += 32) {
    const double x = r0 + lane < mine ? run_sum[r0 + lane] : 0.0;
    const double pre = warp_scan(x);
    const uint32_t some = __ballot_sync(0xffffffffu, x > 0.0);
    const uint32_t hits = __ballot_sync(0xffffffffu, x > 0.0 && c + pre > target);
    if (some) {
      const int l = hits ? __ffs(hits) - 1 : 31 - __clz(some);
      pick = r0 + l;
      at = c + __shfl_sync(0xffffffffu, pre - x, l);
    }
    if (hits) break;
    c += __shfl_sync(0xffffffffu, pre, 31);
  }
  // and that run's entries, in index order: the lanes' first quadruples, then
  // their second
  const int v0 = (r_beg + pick) * RUN;
  float pa[8], qa[8];
  double x[8];
  w.load(v0, pa, qa);
  w.weigh(v0, pa, qa, x);
  c = at;
  int token = -1;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const double s01 = x[4 * h] + x[4 * h + 1], s = s01 + (x[4 * h + 2] + x[4 * h + 3]);
    const double pre = warp_scan(s), base = c + (pre - s);
    const double run[4] = {base + x[4 * h], base + s01, base + (s01 + x[4 * h + 2]), base + s};
    int hit = -1, lastp = -1;
#pragma unroll
    for (int k = 3; k >= 0; --k)
      if (x[4 * h + k] > 0.0 && run[k] > target) hit = v0 + 128 * h + 4 * lane + k - w.shift;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (x[4 * h + k] > 0.0) lastp = v0 + 128 * h + 4 * lane + k - w.shift;
    const uint32_t hits = __ballot_sync(0xffffffffu, hit >= 0), some = __ballot_sync(0xffffffffu, lastp >= 0);
    if (hits) {
      token = __shfl_sync(0xffffffffu, hit, __ffs(hits) - 1);
      break;
    }
    // no entry passes (rounding): the last one with weight
    if (some) token = __shfl_sync(0xffffffffu, lastp, 31 - __clz(some));
    c += __shfl_sync(0xffffffffu, pre, 31);
  }
  if (lane == 0) a.next_token[b] = token;
}

}  // namespace vfy

cudaError_t launch_verify(const VerifyArgs& a, int sms, cudaStream_t st) {
  // A block of the cluster per 4096 entries, up to 16, or 8 or 4 where more a
  // sequence would not all be resident: 5 sequences of 123745 entries take 9.3 us
  // with 8 blocks and 7.5 with 16, one of 32000 6.2 with 4 and 5.6 with 8; 96 of
  // 131072 take 21.2 with 4 (23.2 with 3) and 25.0 with 8, whose last clusters
  // start when the first are through.  With small vocabularies more blocks would
  // only wait.  (Four or more also keep a block's notes within its shared memory.)
  int most = vfy::MAXCL;
  while (most > 4 && (int64_t)a.B * most > (int64_t)vfy::BLOCKS * sms) most /= 2;
  int cl = (a.V + 4095) / 4096;
  cl = cl < most ? cl : most;
  if (cl > 8) {  // past the portable size: allowed once per device
    static std::atomic<uint64_t> done_mask{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64 || !(done_mask & (1ull << dev))) {
      e = cudaFuncSetAttribute(vfy::verify_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
      if (e != cudaSuccess) return e;
      if (dev < 64) done_mask |= 1ull << dev;
    }
  }
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)cl;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.B * (unsigned)cl);
  cfg.blockDim = dim3(vfy::NT);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, vfy::verify_kernel, a);
}

}  // namespace mtla
