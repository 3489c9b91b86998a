// Verification of drafted tokens against the target's probabilities, from given
// random numbers (speculative sampling).
//
// Draft x, drawn from q, is kept with probability min(1, p(x) / q(x)): iff
// u q(x) < p(x).  At the first draft dropped, the next token comes from the
// residual max(p - q, 0), so that kept and drawn tokens together follow p; when
// all are kept, from p of the chunk's last row.  It is drawn by inversion: the
// lowest index whose running sum exceeds u times the sum.
//
// A cluster of CL blocks takes a sequence: only one row of p and of q is read
// (the drafts' probabilities are gathers), so the vocabulary is split over the
// cluster for its latency and bandwidth, and the blocks exchange their sums
// through distributed shared memory.  A warp sums 1024 entries at a time and
// notes each sum; after the exchange the one block that holds the drawn index
// reads one such run again and scans it.  Sums are in double precision: the
// running sum over 10^5 entries of size 10^-5 must place the border between
// neighbours, which 24 bits would miss once in a hundred draws.  Bound by the
// two rows' HBM reads (large batches) or by the chain of four dependent reads
// (small ones).
#include <cooperative_groups.h>

#include "paged.cuh"

namespace mtla {
namespace vfy {

namespace cg = cooperative_groups;
constexpr int CL = 8;
constexpr int NT = 256, NW = NT / 32;
constexpr int RUN = 1024;                           // entries a warp sums at a time
constexpr int MAXV = 1 << 24;
constexpr int MAXRUNS = MAXV / RUN / CL;            // runs of a block: 2048

// entries that are NaN, infinite or not above zero count as zero
__device__ __forceinline__ float clean(float x) { return x > 0.f && x <= 3.4028234663852886e38f ? x : 0.f; }

__global__ void __cluster_dims__(CL, 1, 1) __launch_bounds__(NT) verify_kernel(const VerifyArgs a) {
  cg::cluster_group cluster = cg::this_cluster();
  __shared__ double run_sum[MAXRUNS];
  __shared__ double my_total, all[CL];
  __shared__ int first_drop, pick;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = (int)cluster.block_rank(), b = blockIdx.x / CL;

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
  // ---- the first draft dropped (n - 1: none); every block finds it for itself
  if (tid == 0) first_drop = n - 1;
  __syncthreads();
  for (int i0 = 0; i0 < n - 1; i0 += NT) {
    const int i = i0 + tid;
    if (i < n - 1) {
      const int64_t row = first + i;
      const int x = a.tokens[row + 1];
      bool keep = false;
      if (x >= 0 && x < a.V) {
        const double p = clean(a.p[row * a.ld_p + x]), q = a.q ? clean(a.q[row * a.ld_q + x]) : 1.f;
        keep = (double)a.u_accept[row] * q < p;
      } else if (rank == 0) {
        set_err(a.dev_err, MTLA_DEVERR_TOKEN);
      }
      if (!keep) atomicMin(&first_drop, i);
    }
    __syncthreads();
    if (first_drop < i0 + NT) break;
  }
  const int drop = first_drop;
  const float* pr = a.p + (int64_t)(first + drop) * a.ld_p;
  const float* qr = a.q ? a.q + (int64_t)(first + drop) * a.ld_q : nullptr;
  // certain drafts (no q): the residual is p without the dropped token
  const int hole = !a.q && drop < n - 1 ? a.tokens[first + drop + 1] : -1;
  bool residual = drop < n - 1;

  const int runs = (a.V + RUN - 1) / RUN, per = (runs + CL - 1) / CL;
  const int r_beg = rank * per < runs ? rank * per : runs, r_end = r_beg + per < runs ? r_beg + per : runs;
  auto weight = [&](int v) -> double {
    const double p = clean(pr[v]);
    if (!residual) return p;
    if (qr) {
      const double d = p - (double)clean(qr[v]);
      return d > 0.0 ? d : 0.0;
    }
    return v == hole ? 0.0 : p;
  };
  double total = 0.0;
  for (;;) {
    for (int r = r_beg + warp; r < r_end; r += NW) {
      double sum = 0.0;
      const int v0 = r * RUN + lane;
#pragma unroll 8
      for (int k = 0; k < RUN / 32; ++k) {
        const int v = v0 + 32 * k;
        if (v < a.V) sum += weight(v);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      if (lane == 0) run_sum[r - r_beg] = sum;
    }
    __syncthreads();
    if (warp == 0) {
      double sum = 0.0;
      for (int r = lane; r < r_end - r_beg; r += 32) sum += run_sum[r];
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      if (lane == 0) my_total = sum;
    }
    cluster.sync();
    if (tid < CL) all[tid] = *cluster.map_shared_rank(&my_total, tid);
    cluster.sync();  // every block has read the totals: they may be written again, and blocks may leave
    total = 0.0;
    for (int r = 0; r < CL; ++r) total += all[r];
    if (total > 0.0 || !residual) break;
    residual = false;  // nothing above q: draw from p
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
  const float u = a.u_sample[b];
  const double target = (u > 0.f ? (double)u : 0.0) * total;
  int owner = -1;
  double before = 0.0;
  {
    double c = 0.0;
    for (int r = 0; r < CL; ++r) {
      if (all[r] > 0.0) {
        // (the last block with any weight takes what rounding leaves over)
        owner = r;
        before = c;
        if (c + all[r] > target) break;
      }
      c += all[r];
    }
  }
  if (owner != rank) return;
  if (tid == 0) {
    double c = before;
    int at = -1;
    for (int r = 0; r < r_end - r_beg; ++r) {
      if (run_sum[r] > 0.0) {
        at = r;
        before = c;
        if (c + run_sum[r] > target) break;
      }
      c += run_sum[r];
    }
    pick = at;
    my_total = before;
  }
  __syncthreads();
  if (warp != 0) return;
  // warp 0 scans the run: lane l holds entries 32 l .. 32 l + 31
  const int v0 = (r_beg + pick) * RUN + 32 * lane;
  before = my_total;
  double w[32], sum = 0.0;
#pragma unroll
  for (int k = 0; k < 32; ++k) {
    w[k] = v0 + k < a.V ? weight(v0 + k) : 0.0;
    sum += w[k];
  }
  double pre = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const double v = __shfl_up_sync(0xffffffffu, pre, o);
    if (lane >= o) pre += v;
  }
  double c = before + (pre - sum);
  int hit = -1, lastp = -1;
#pragma unroll
  for (int k = 0; k < 32; ++k) {
    c += w[k];
    if (w[k] > 0.0) lastp = v0 + k;
    if (hit < 0 && c > target && w[k] > 0.0) hit = v0 + k;
  }
  const uint32_t hits = __ballot_sync(0xffffffffu, hit >= 0), some = __ballot_sync(0xffffffffu, lastp >= 0);
  // no entry passes (rounding): the last one with weight
  if (hits ? lane == __ffs(hits) - 1 : lane == 31 - __clz(some)) a.next_token[b] = hits ? hit : lastp;
}

}  // namespace vfy

cudaError_t launch_verify(const VerifyArgs& a, cudaStream_t st) {
  vfy::verify_kernel<<<(unsigned)a.B * vfy::CL, vfy::NT, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace mtla
