// moe.cu -- tokens sorted by expert and brought back: the T x k expert choices
// as one stable order by expert (what the experts' products in gemv_fused.cu
// and prefill.cu walk), and the weighted sum of the experts' outputs per token.
//
// Sort: a counting sort.  The T * k choices are cut into chunks, one CTA each,
// which counts its chunk's experts, adds up the counts of all chunks (every CTA
// for itself), scans them over the experts, and gives each choice its place:
// expert start + the same expert's choices in earlier chunks + in earlier warps
// of this chunk + in earlier lanes.  No atomics decide an order, so the sort is
// stable and repeatable.  Bound by latency.  A decode step is one CTA; up to
// kSortClusterChoices choices are one cluster, whose CTAs read each other's counts
// from shared memory (2048 x 4 choices of 16 experts: 6.0 us with two launches, 4.8
// so); beyond that a first kernel counts.
//
// Back: out[t] = residual[t] + sum_j weight[t][j] * y[pos[t][j]], j in order,
// fp32.  HBM bound: each chosen row is read once; a thread holds one vector of a
// token's output and has the loads of up to 8 rows in flight.
#include "dsq_device.cuh"
#include "dsq_host.h"

namespace dsq {
namespace {

constexpr int kSortMaxE = 1024;
constexpr int kSortThreads = 512;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int64_t kSortChunk = 2048;
constexpr int64_t kSortMaxChunks = 128;

constexpr int kSortCluster = 8;
constexpr int64_t kSortClusterChoices = kSortCluster * kSortChunk;

// Choices per chunk: at least kSortChunk, and few enough chunks that adding
// up their counts stays short.
int64_t sort_chunk(int64_t n) {
  const int64_t even = (n + kSortMaxChunks - 1) / kSortMaxChunks;
  return even > kSortChunk ? even : kSortChunk;
}

__global__ void __launch_bounds__(kSortThreads) sort_count_kernel(const int32_t *expert, int64_t n, int64_t chunk,
                                                                  int E, int32_t *counts) {
  __shared__ int32_t c[kSortMaxE];
  pdl_trigger();
  for (int e = threadIdx.x; e < E; e += kSortThreads) c[e] = 0;
  pdl_wait();
  __syncthreads();
  const int64_t lo = blockIdx.x * chunk, hi = lo + chunk < n ? lo + chunk : n;
  for (int64_t i = lo + threadIdx.x; i < hi; i += kSortThreads) {
    const int e = expert[i];
    if (e >= 0 && e < E) atomicAdd(&c[e], 1);   // a count: the order does not matter
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += kSortThreads) counts[blockIdx.x * static_cast<int64_t>(E) + e] = c[e];
}

// Where the counts of all chunks come from: there is one chunk, the CTAs are one
// cluster, or the kernel before counted (counts: [chunks][E]).
enum : int { kSortOne = 0, kSortInCluster = 1, kSortCounted = 2 };
template <int MODE>
__global__ void __launch_bounds__(kSortThreads) sort_place_kernel(const int32_t *expert, int64_t n, int64_t chunk,
                                                                  int chunks, int E, const int32_t *counts,
                                                                  int32_t *offsets, int32_t *rows, int32_t *pos) {
  constexpr bool CLUSTER = MODE == kSortInCluster, COUNTED = MODE == kSortCounted;
  extern __shared__ int32_t table[];   // [kSortWarps][E]: first the warps' counts, then their next places
  __shared__ int32_t start[kSortMaxE + 1], scan[kSortWarps], own[CLUSTER ? kSortMaxE : 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_trigger();
  for (int i = threadIdx.x; i < kSortWarps * E; i += kSortThreads) table[i] = 0;
  pdl_wait();
  __syncthreads();
  const int64_t lo = blockIdx.x * chunk, hi = lo + chunk < n ? lo + chunk : n;
  // each warp owns a contiguous part of the chunk, whole groups of 32
  const int64_t part = ((chunk + kSortWarps - 1) / kSortWarps + 31) / 32 * 32;
  const int64_t wlo = lo + warp * part, whi = wlo + part < hi ? wlo + part : hi;
  int32_t *mine = table + warp * E;
  // kAhead choices of a lane are loaded at once, all of them up to one cluster's,
  // and stay in registers for the second pass (2048 x 6 choices of 64: 6.2 -> 5.3
  // us).  Beyond, a warp's many turns go faster one load at a time, and the table is
  // read only where it is rewritten (8192 x 4 of 64: 8.4 us in the clusters' form,
  // 7.6 so; 40,000 x 8: 26.5 and 16.3; 400,000 x 8: 75.9 and 69.1).
  constexpr int kAhead = COUNTED ? 1 : static_cast<int>(kSortChunk) / kSortThreads;
  int ex[kAhead];
  auto load = [&](int64_t i0) {
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int64_t i = i0 + j * 32 + lane;
      ex[j] = i < whi ? expert[i] : -1;
      if (ex[j] >= E) ex[j] = -1;
    }
  };
  for (int64_t i0 = wlo; i0 < whi; i0 += 32 * kAhead) {
    load(i0);
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
      if (ex[j] >= 0) atomicAdd(&mine[ex[j]], 1);
  }
  __syncthreads();
  // totals over all chunks, and over the chunks before this one (kept in before[])
  constexpr int kPer = kSortMaxE / kSortThreads;
  int32_t total[kPer], before[kPer], held[COUNTED ? 1 : kPer][kSortWarps];
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int e = static_cast<int>(threadIdx.x) * kPer + j;
    total[j] = before[j] = 0;
    if (e >= E || COUNTED) continue;
#pragma unroll
    for (int w = 0; w < kSortWarps; ++w) held[COUNTED ? 0 : j][w] = table[w * E + e];
#pragma unroll
    for (int w = 0; w < kSortWarps; ++w) total[j] += held[COUNTED ? 0 : j][w];
    if (CLUSTER) own[e] = total[j];
  }
  if constexpr (CLUSTER) cluster_sync();   // every CTA's own[] is written
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int e = static_cast<int>(threadIdx.x) * kPer + j;
    if (e >= E || MODE == kSortOne) continue;
    total[j] = 0;
    if constexpr (CLUSTER) {
      const uint32_t at = smem_u32(&own[e]);
      int32_t v[kSortCluster];
#pragma unroll
      for (int c = 0; c < kSortCluster; ++c) v[c] = static_cast<int32_t>(ld_shared_remote_u32(mapa_shared(at, static_cast<uint32_t>(c))));
#pragma unroll
      for (int c = 0; c < kSortCluster; ++c) {
        total[j] += v[c];
        if (c < static_cast<int>(blockIdx.x)) before[j] += v[c];
      }
    } else {
#pragma unroll 8
      for (int c = 0; c < chunks; ++c) {
        const int32_t v = counts[static_cast<int64_t>(c) * E + e];
        total[j] += v;
        if (c < static_cast<int>(blockIdx.x)) before[j] += v;
      }
    }
  }
  if constexpr (CLUSTER) cluster_arrive();   // done with the others' counts
  // exclusive scan over the experts (thread order = expert order)
  int32_t sum = 0;
#pragma unroll
  for (int j = 0; j < kPer; ++j) sum += total[j];
  int32_t inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int32_t up = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += up;
  }
  if (lane == 31) scan[warp] = inc;
  __syncthreads();
  int32_t base = inc - sum;
  for (int w = 0; w < warp; ++w) base += scan[w];
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int e = static_cast<int>(threadIdx.x) * kPer + j;
    if (e < E) {
      start[e] = base;
      int32_t next = base + before[j];   // where this chunk's choices of e begin
      if constexpr (COUNTED)
#pragma unroll
        for (int w = 0; w < kSortWarps; ++w) held[0][w] = table[w * E + e];
#pragma unroll
      for (int w = 0; w < kSortWarps; ++w) {
        table[w * E + e] = next;
        next += held[COUNTED ? 0 : j][w];
      }
    }
    base += total[j];
    if (e == E - 1) start[E] = base;
  }
  __syncthreads();
  if (blockIdx.x == 0)
    for (int e = threadIdx.x; e <= E; e += kSortThreads) offsets[e] = start[e];
  const int64_t kept = start[E];
  for (int64_t i0 = wlo; i0 < whi; i0 += 32 * kAhead) {
    if (COUNTED) load(i0);
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int64_t i = i0 + j * 32 + lane;
      const int e = ex[j];
      const unsigned same = __match_any_sync(0xffffffffu, e);
      const int rank = __popc(same & ((1u << lane) - 1u));
      int32_t p = -1;
      if (e >= 0) p = mine[e] + rank;
      __syncwarp();
      if (e >= 0) {
        if (rank == 0) mine[e] = p + __popc(same);
        rows[p] = static_cast<int32_t>(i);
      }
      __syncwarp();
      if (i < whi) pos[i] = p;
    }
  }
  // the places that no choice took
  for (int64_t p = lo + threadIdx.x; p < hi; p += kSortThreads)
    if (p >= kept) rows[p] = -1;
  if constexpr (CLUSTER) cluster_wait();   // no CTA leaves while another may still read its counts
}

template <int V> struct MoeVec;
template <> struct MoeVec<1> { using T = float; };
template <> struct MoeVec<4> { using T = float4; };

constexpr int kBackThreads = 128;

// FLIGHT rows' loads are in flight together: k of them where k is at most 8 (2048
// tokens, N = 4096: k = 6 42.9 us with 6, 44.7 with 8; k = 2 24.9 with 4, 31.1
// with 8 -- the slots past k cost registers and so residency).  y is read once and
// out not again here, so both are streamed past L2's other contents.  pos and
// weight come from kernels just before: plain loads, since a read-only load may
// be moved above the wait for them.  The residual's load follows the rows' (in
// front of the positions 51.3 us with the sort, behind 49.8).
template <int V, int FLIGHT>
__global__ void __launch_bounds__(kBackThreads) combine_kernel(const float *y, int64_t P, const int32_t *pos,
                                                               const float *weight, const float *residual, int k,
                                                               int64_t N, float *out) {
  using T = typename MoeVec<V>::T;
  pdl_trigger();
  pdl_wait();
  const int64_t row = blockIdx.x;
  const int64_t col = (blockIdx.y * static_cast<int64_t>(kBackThreads) + threadIdx.x) * V;
  if (col >= N) return;
  const T zero{};
  T res = zero;
  float sum[V];
#pragma unroll
  for (int e = 0; e < V; ++e) sum[e] = 0.0f;
  for (int j0 = 0; j0 < k; j0 += FLIGHT) {
    T v[FLIGHT];
    float w[FLIGHT];
    int32_t p[FLIGHT];
#pragma unroll
    for (int j = 0; j < FLIGHT; ++j) {
      p[j] = -1;
      w[j] = 1.0f;
      if (j0 + j < k) {
        p[j] = pos[row * k + j0 + j];
        if (weight) w[j] = weight[row * k + j0 + j];
      }
    }
#pragma unroll
    for (int j = 0; j < FLIGHT; ++j)
      if (p[j] >= 0 && p[j] < P) v[j] = __ldcs(reinterpret_cast<const T *>(y + p[j] * N + col));
    if (residual && j0 == 0) res = *reinterpret_cast<const T *>(residual + row * N + col);
#pragma unroll
    for (int j = 0; j < FLIGHT; ++j)
      if (p[j] >= 0 && p[j] < P) {
#pragma unroll
        for (int e = 0; e < V; ++e)
          sum[e] = __fadd_rn(sum[e], __fmul_rn(w[j], reinterpret_cast<const float *>(&v[j])[e]));
      }
  }
  T o;
#pragma unroll
  for (int e = 0; e < V; ++e)
    reinterpret_cast<float *>(&o)[e] = residual ? __fadd_rn(reinterpret_cast<const float *>(&res)[e], sum[e]) : sum[e];
  __stcs(reinterpret_cast<T *>(out + row * N + col), o);
}

template <int V>
cudaError_t combine_launch(dim3 grid, cudaStream_t st, const float *y, int64_t P, const int32_t *pos,
                           const float *weight, const float *residual, int k, int64_t N, float *out) {
  const dim3 block(kBackThreads);
  if (k == 1) return launch_pdl(combine_kernel<V, 1>, grid, block, 0, st, y, P, pos, weight, residual, k, N, out);
  if (k == 2) return launch_pdl(combine_kernel<V, 2>, grid, block, 0, st, y, P, pos, weight, residual, k, N, out);
  if (k <= 4) return launch_pdl(combine_kernel<V, 4>, grid, block, 0, st, y, P, pos, weight, residual, k, N, out);
  if (k <= 6) return launch_pdl(combine_kernel<V, 6>, grid, block, 0, st, y, P, pos, weight, residual, k, N, out);
  return launch_pdl(combine_kernel<V, 8>, grid, block, 0, st, y, P, pos, weight, residual, k, N, out);
}

}  // namespace
}  // namespace dsq

extern "C" size_t dsq_moe_sort_workspace_bytes(int64_t T, int64_t k, int64_t E) {
  if (T < 0 || k < 1 || E < 1 || E > dsq::kSortMaxE || T > (int64_t(1) << 30) / k) return 0;
  const int64_t n = T * k, chunk = dsq::sort_chunk(n), chunks = (n + chunk - 1) / chunk;
  return chunks <= 1 ? 0 : static_cast<size_t>(chunks) * E * sizeof(int32_t);
}

extern "C" int dsq_moe_sort(const int32_t *expert, int64_t T, int64_t k, int64_t E, int32_t *offsets, int32_t *rows,
                            int32_t *pos, void *workspace, size_t workspace_bytes, void *stream) {
  using namespace dsq;
  DSQ_REQUIRE(T >= 0 && k >= 1 && E >= 1, DSQ_ERR_INVALID_ARG, "dsq_moe_sort: T=%lld k=%lld E=%lld", (long long)T,
              (long long)k, (long long)E);
  DSQ_REQUIRE(E <= kSortMaxE && T <= (int64_t(1) << 30) / k, DSQ_ERR_SHAPE,
              "dsq_moe_sort: size out of range (E <= %d, T*k <= 2^30)", kSortMaxE);
  DSQ_REQUIRE(offsets && (T == 0 || (expert && rows && pos)), DSQ_ERR_INVALID_ARG, "dsq_moe_sort: null pointer");
  DSQ_REQUIRE(aligned(expert, 4) && aligned(offsets, 4) && aligned(rows, 4) && aligned(pos, 4), DSQ_ERR_ALIGNMENT,
              "dsq_moe_sort: pointers must be 4-byte aligned");
  const size_t need = dsq_moe_sort_workspace_bytes(T, k, E);
  DSQ_REQUIRE(need == 0 || (workspace && workspace_bytes >= need), DSQ_ERR_WORKSPACE,
              "dsq_moe_sort: workspace of %zu bytes needed, %zu given", need, workspace_bytes);
  DSQ_REQUIRE(need == 0 || aligned(workspace, 256), DSQ_ERR_ALIGNMENT,
              "dsq_moe_sort: workspace must be 256-byte aligned");
  int rc = device_ready(nullptr, nullptr);
  if (rc != DSQ_OK) return rc;
  cudaStream_t st = as_stream(stream);
  const int64_t n = T * k;
  const bool cluster = n > kSortChunk && n <= kSortClusterChoices;
  const int64_t chunk = cluster ? (n + kSortCluster - 1) / kSortCluster : sort_chunk(n);
  const int chunks = cluster ? kSortCluster : n == 0 ? 1 : static_cast<int>((n + chunk - 1) / chunk);
  int32_t *counts = static_cast<int32_t *>(workspace);
  const int Ei = static_cast<int>(E);
  if (chunks > 1 && !cluster) {
    const cudaError_t e = launch_pdl(sort_count_kernel, dim3(static_cast<unsigned>(chunks)), dim3(kSortThreads), 0, st,
                                     expert, n, chunk, Ei, counts);
    if (e != cudaSuccess) return fail(DSQ_ERR_LAUNCH, "dsq_moe_sort: count: %s", cudaGetErrorString(e));
    rc = after_launch("dsq_moe_sort: count");
    if (rc != DSQ_OK) return rc;
  }
  const size_t smem = static_cast<size_t>(kSortWarps) * E * sizeof(int32_t);
  const auto kern = cluster       ? sort_place_kernel<kSortInCluster>
                    : chunks == 1 ? sort_place_kernel<kSortOne>
                                  : sort_place_kernel<kSortCounted>;
  rc = set_smem_once(reinterpret_cast<const void *>(kern), static_cast<int>(kSortWarps * kSortMaxE * sizeof(int32_t)),
                     "dsq_moe_sort");
  if (rc != DSQ_OK) return rc;
  const cudaError_t e = launch_pdl_cluster(kern, cluster ? kSortCluster : 1u, dim3(static_cast<unsigned>(chunks)),
                                           dim3(kSortThreads), smem, st, expert, n, chunk, chunks, Ei,
                                           static_cast<const int32_t *>(counts), offsets, rows, pos);
  if (e != cudaSuccess) return fail(DSQ_ERR_LAUNCH, "dsq_moe_sort: %s", cudaGetErrorString(e));
  return after_launch("dsq_moe_sort");
}

extern "C" int dsq_moe_combine(const float *y, int64_t P, const int32_t *pos, const float *weight,
                               const float *residual, int64_t T, int64_t k, int64_t N, float *out, void *stream) {
  using namespace dsq;
  DSQ_REQUIRE(T >= 0 && k >= 1 && N >= 1 && P >= 0, DSQ_ERR_INVALID_ARG, "dsq_moe_combine: T=%lld k=%lld N=%lld P=%lld",
              (long long)T, (long long)k, (long long)N, (long long)P);
  DSQ_REQUIRE(T < (int64_t(1) << 31) && k <= 1024 && N <= (int64_t(1) << 24) && P < (int64_t(1) << 31),
              DSQ_ERR_SHAPE, "dsq_moe_combine: size out of range (k <= 1024, N <= 2^24)");
  if (T == 0) return DSQ_OK;
  DSQ_REQUIRE(pos && out && (y || P == 0), DSQ_ERR_INVALID_ARG, "dsq_moe_combine: null pointer");
  DSQ_REQUIRE(aligned(y, 16) && aligned(residual, 16) && aligned(out, 16) && aligned(pos, 4) && aligned(weight, 4),
              DSQ_ERR_ALIGNMENT, "dsq_moe_combine: y, residual and out must be 16-byte aligned");
  int rc = device_ready(nullptr, nullptr);
  if (rc != DSQ_OK) return rc;
  const int V = N % 4 == 0 ? 4 : 1;
  const dim3 grid(static_cast<unsigned>(T), static_cast<unsigned>((N / V + kBackThreads - 1) / kBackThreads));
  DSQ_REQUIRE(grid.y <= 65535u, DSQ_ERR_SHAPE, "dsq_moe_combine: N=%lld out of range", (long long)N);
  cudaStream_t st = as_stream(stream);
  const int ki = static_cast<int>(k);
  const cudaError_t e = V == 4 ? combine_launch<4>(grid, st, y, P, pos, weight, residual, ki, N, out)
                               : combine_launch<1>(grid, st, y, P, pos, weight, residual, ki, N, out);
  if (e != cudaSuccess) return fail(DSQ_ERR_LAUNCH, "dsq_moe_combine: %s", cudaGetErrorString(e));
  return after_launch("dsq_moe_combine");
}
