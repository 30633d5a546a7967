// gemv_rows.cuh -- the one-token form of the fused decode products
// (gemv_fused.cu): whole weight rows instead of 32-row boxes.
//
// A lane owns one 256-element unit of a row and keeps that unit's activation
// slice in registers for all rows; G lanes (units per row, rounded up to a
// power of two) share a row, so a warp takes 32 / G rows at a time.  They arrive
// as one contiguous bulk copy per weight -- of a gate / up pair the rows of both,
// half the lanes each -- into the warp's own ring of slots; the lanes' sums meet
// in xor-shuffles (the single-token GEMV's order, so the sums are its own bit
// for bit), and the row's first lane applies the epilogue.  No warp waits for
// another.  It streams faster than the boxes wherever there are many rows:
// a box costs the copy engine about 11 cycles for each of its rows however
// short, and a Q4_K unit is only 144 bytes.
#pragma once

#include "epilogue.cuh"
#include "units.cuh"

namespace dsq {
namespace {

constexpr int kRowsMaxE = 1024;

struct RowsArgs {
  const uint8_t *w[2];
  float *y;
  const float *bias[2];
  const float *residual;
  int act;
  int64_t N, K, row_bytes;
  int nunits;            // K / 256 <= 32
  int per;               // slots of a weight: ceil(N / outputs of a slot)
  int stages, slot_bytes;
  const int8_t *xq;
  const float *xd;
  const int32_t *xs;
  const int32_t *offsets, *rows;   // experts (as in FusedArgs)
  int E, k, P;
  int64_t A;
  WaitCtl wait;
};

// Passes a lane makes over a slot: two rows' units side by side hide more of a
// Q4_K unit's unpacking and share the slot's waits.
__host__ __device__ constexpr int rows_mult(int type, int G, bool gated) {
  return type == DSQ_Q4_K && !(gated && G == 32) ? 2 : 1;
}

// A warp's place: sorted row p (0 for a plain product) of expert e, slot s of its
// weight.
struct RowsCursor {
  int p, e, s;
};

template <int TYPE, int G, bool GATED, bool EXPERTS, int NW>
__global__ void __launch_bounds__(NW * 32, 1) gemv_rows_kernel(const __grid_constant__ RowsArgs a) {
  constexpr int UB = Unit<TYPE>::kBytes;
  constexpr int R = 32 / G;                             // rows of a pass
  constexpr int PASSES = GATED && G == 32 ? 2 : 1;      // a pair of rows longer than half a warp: one after the other
  constexpr int EACH = GATED && G < 32 ? R / 2 : R;     // outputs of a pass
  constexpr int MULT = rows_mult(TYPE, G, GATED);       // passes over the slot's outputs
  constexpr int OUT = EACH * MULT;                      // outputs of a slot
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = lane / G, j = lane % G;
  const int out0 = sub % EACH;              // this lane's first output within the slot
  const int seg = GATED && G < 32 ? sub / EACH : 0;
  const int S = a.stages;
  uint8_t *ring = smem + static_cast<size_t>(warp) * S * a.slot_bytes;
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + static_cast<size_t>(NW) * S * a.slot_bytes) + warp * S;
  int32_t *off = nullptr;
  if constexpr (EXPERTS) {
    __shared__ int32_t shared_off[kRowsMaxE + 1];
    off = shared_off;
  }
  if (lane == 0) {
    for (int s = 0; s < S; ++s) mbar_init(&bars[s], 1);
    fence_barrier_init();
  }
  __syncwarp();   // the other lanes wait on these barriers: not before they exist
  const uint64_t policy = l2_policy_evict_first();
  int total = a.per;
  [[maybe_unused]] int32_t choice = -1;   // rows[lane], looked up ahead
  uint32_t lo, hi;   // this CTA's slots; its warps take them in turn
  auto share = [&]() {
    const uint32_t n = static_cast<uint32_t>(total), each = n / gridDim.x, more = n - each * gridDim.x;
    lo = each * blockIdx.x + min(blockIdx.x, more);
    hi = lo + each + (blockIdx.x < more ? 1u : 0u);
  };
  auto at = [&](uint32_t it) {
    RowsCursor c{0, 0, static_cast<int>(it)};
    if constexpr (EXPERTS) {
      c.p = static_cast<int>(it / static_cast<uint32_t>(a.per));
      c.s = static_cast<int>(it) - c.p * a.per;
      int x = 0, y = a.E;   // the last expert that starts at or before p
      while (y - x > 1) {
        const int mid = (x + y) >> 1;
        if (off[mid] <= c.p) x = mid;
        else y = mid;
      }
      c.e = x;
    }
    return c;
  };
  auto step = [&](RowsCursor &c) {
    c.s += NW;
    if constexpr (EXPERTS) {
      while (c.s >= a.per) {
        c.s -= a.per;
        ++c.p;
        while (c.e + 1 < a.E && off[c.e + 1] <= c.p) ++c.e;
      }
    }
  };
  // rows of the slot that exist, and where they start in a weight
  auto rows_of = [&](const RowsCursor &c) { return static_cast<int>(min(static_cast<int64_t>(OUT), a.N - static_cast<int64_t>(c.s) * OUT)); };
  auto first_byte = [&](const RowsCursor &c) {
    return ((EXPERTS ? c.e * a.N : 0) + static_cast<int64_t>(c.s) * OUT) * a.row_bytes;
  };
  if constexpr (!EXPERTS) {
    // weights are read-only: this warp's first slots toward L2 while the
    // kernel before us finishes
    share();
    if (lane == 0) {
      for (int s = 0; s < S && lo + warp + s * NW < hi; ++s) {
        const RowsCursor c = at(lo + warp + s * NW);
        const uint32_t bytes = static_cast<uint32_t>(rows_of(c) * a.row_bytes);
        prefetch_l2(a.w[0] + first_byte(c), bytes);
        if (GATED) prefetch_l2(a.w[1] + first_byte(c), bytes);
      }
    }
  }
  pdl_trigger();
  pdl_wait();
  if constexpr (EXPERTS) {
    // rows holds the sorted rows there are, which may be fewer than P.  A warp's
    // lanes keep the first 32 (in shared memory, behind a barrier: 16.6 against 16.1 us)
    const int listed = min(a.offsets[a.E], a.P);
    for (int e = threadIdx.x; e <= a.E; e += NW * 32) off[e] = min(max(a.offsets[e], 0), a.P);
    if (a.rows && lane < listed) choice = a.rows[lane];
    __syncthreads();
    total = off[a.E] * a.per;
    share();
  }
  const uint32_t first = lo + warp;
  if (first >= hi) return;
  const int mine = static_cast<int>((hi - first + NW - 1) / NW);
  RowsCursor next = at(first), c = next;
  auto issue = [&](int s) {
    uint8_t *dst = ring + static_cast<size_t>(s) * a.slot_bytes;
    const uint32_t bytes = static_cast<uint32_t>(rows_of(next) * a.row_bytes);
    mbar_arrive_expect_tx(&bars[s], GATED ? 2 * bytes : bytes);
    bulk_g2s(dst, a.w[0] + first_byte(next), bytes, &bars[s], policy);
    if (GATED) bulk_g2s(dst + OUT * a.row_bytes, a.w[1] + first_byte(next), bytes, &bars[s], policy);
    step(next);
  };
  if (lane == 0)
    for (int s = 0; s < S && s < mine; ++s) issue(s);
  ActSlice act;
  int64_t have = -2;   // activation row whose slices the lanes hold (-1: zeros)
  int at_p = -1;       // the sorted row it was last looked up for
  int slot = 0;
  uint32_t parity = 0;
  for (int it = 0; it < mine; ++it, step(c)) {
    int64_t src = have;
    if (c.p != at_p) {
      at_p = c.p;
      src = 0;
      if constexpr (EXPERTS) {
        src = c.p;
        if (a.rows) {
          const int32_t f = c.p < 32 ? __shfl_sync(0xffffffffu, choice, c.p) : a.rows[c.p];
          src = f < 0 ? -1 : f / a.k;
        }
        if (src >= a.A) src = -1;
      }
    }
    if (src != have) {   // the sorted rows of one token keep their slices
      have = src;
      if (src >= 0 && j < a.nunits) {
        const int64_t e0 = src * a.K + j * 256;
        load_act<TYPE>(act, a.xq + e0, a.xd + e0 / 32, TYPE == DSQ_Q4_K ? a.xs + e0 / 32 : nullptr);
      } else {
#pragma unroll
        for (int i = 0; i < 64; ++i) act.q[i] = 0u;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          act.d[i] = 0.0f;
          act.s[i] = 0;
        }
      }
    }
    const int rows = rows_of(c);
    const int64_t n0 = static_cast<int64_t>(c.s) * OUT + out0;
    const int64_t brow = (EXPERTS ? c.e * a.N : 0) + n0;
    const int64_t yrow = static_cast<int64_t>(c.p) * a.N + n0;
    // what the epilogue reads, under way before the weights are waited for
    float b0[MULT], b1 = 0.0f, res[MULT];
#pragma unroll
    for (int m = 0; m < MULT; ++m) {
      b0[m] = res[m] = 0.0f;
      if (j == 0 && out0 + m * EACH < rows) {
        if (a.bias[seg]) b0[m] = a.bias[seg][brow + m * EACH];
        if (PASSES == 2 && a.bias[1]) b1 = a.bias[1][brow];
        if (a.residual && seg == 0) res[m] = a.residual[yrow + m * EACH];
      }
    }
    const bool ok = __all_sync(0xffffffffu, mbar_wait_for(&bars[slot], parity, a.wait.limit_ns));
    if (!ok) {
      if (lane == 0) {
        record_timeout(a.wait);
        for (int k = it; k < mine && k < it + S; ++k)
          mbar_wait_for(&bars[k % S], static_cast<uint32_t>((k / S) & 1), kDrainLimitNs);
      }
      __syncwarp();
      return;
    }
    const uint8_t *slotp = ring + static_cast<size_t>(slot) * a.slot_bytes;
    constexpr int NACC = PASSES * MULT;
    float acc[NACC];
#pragma unroll
    for (int k = 0; k < NACC; ++k) {
      const int m = PASSES == 2 ? 0 : k;
      acc[k] = 0.0f;
      if (out0 + m * EACH < rows && j < a.nunits) {
        const uint8_t *p =
            slotp + static_cast<size_t>((PASSES == 2 ? k : seg) * OUT + out0 + m * EACH) * a.row_bytes + j * UB;
        int32_t is[8];
        if constexpr (TYPE == DSQ_Q8_0) acc[k] += unit_q8_0<false>(p, act, is);
        else acc[k] += unit_q4_k<false>(p, act, is);
      }
    }
    __syncwarp();
    if (lane == 0 && it + S < mine) {
      fence_proxy_async_smem();
      issue(slot);
    }
#pragma unroll
    for (int o = G / 2; o >= 1; o >>= 1)
#pragma unroll
      for (int k = 0; k < NACC; ++k) acc[k] += __shfl_xor_sync(0xffffffffu, acc[k], o);
#pragma unroll
    for (int m = 0; m < MULT; ++m) {
      float v = acc[m];
      if (a.bias[seg]) v = __fadd_rn(v, b0[m]);
      float up = 0.0f;
      if (GATED) {
        if (PASSES == 2) up = a.bias[1] ? __fadd_rn(acc[NACC - 1], b1) : acc[NACC - 1];
        else up = __shfl_down_sync(0xffffffffu, v, 16);
      }
      if (out0 + m * EACH < rows && j == 0 && seg == 0) {
        v = activate(v, a.act);
        if (GATED) v = __fmul_rn(v, up);
        if (a.residual) v = __fadd_rn(v, res[m]);
        a.y[yrow + m * EACH] = v;
      }
    }
    if (++slot == S) {
      slot = 0;
      parity ^= 1u;
    }
  }
}

using RowsKernel = void (*)(const RowsArgs);
template <int TYPE, int G, int NW>
RowsKernel rows_kernel_g(bool gated, bool experts) {
  if (experts) return gated ? gemv_rows_kernel<TYPE, G, true, true, NW> : gemv_rows_kernel<TYPE, G, false, true, NW>;
  return gated ? gemv_rows_kernel<TYPE, G, true, false, NW> : gemv_rows_kernel<TYPE, G, false, false, NW>;
}
template <int TYPE, int NW>
RowsKernel rows_kernel(int G, bool gated, bool experts) {
  switch (G) {
    case 1: return rows_kernel_g<TYPE, 1, NW>(gated, experts);
    case 2: return rows_kernel_g<TYPE, 2, NW>(gated, experts);
    case 4: return rows_kernel_g<TYPE, 4, NW>(gated, experts);
    case 8: return rows_kernel_g<TYPE, 8, NW>(gated, experts);
    case 16: return rows_kernel_g<TYPE, 16, NW>(gated, experts);
    default: return rows_kernel_g<TYPE, 32, NW>(gated, experts);
  }
}

// Q4_K rows per SM between which 12 warps beat 8 (gate and up weights of 2048 rows
// each, K = 4096: 6 experts, 166 rows an SM, 16.2 against 17.0 us; 12 experts, 332
// rows, 27.1 against 25.5).
constexpr int64_t kRowsMid = 140, kRowsLong = 300;

// Whether the kernel takes the call: a lane per unit, slots counted in 32 bits.
bool rows_fit(int64_t K, int64_t N, int64_t P) { return K <= 32 * 256 && N * P < (int64_t(1) << 30); }

// Launches it for `a` (its shape-dependent part is filled in here); groups:
// sorted rows there can be (1 for a plain product).
int rows_launch(const char *name, int type, RowsArgs &a, bool gated, bool experts, int64_t groups, int sms,
                cudaStream_t st) {
  a.nunits = static_cast<int>(a.K / 256);
  int G = 1;
  while (G < a.nunits) G <<= 1;
  const int R = 32 / G, out = (gated && G < 32 ? R / 2 : R) * rows_mult(type, G, gated);
  a.row_bytes = static_cast<int64_t>(dsq_row_bytes(type, a.K));
  a.per = static_cast<int>((a.N + out - 1) / out);
  a.slot_bytes = static_cast<int>((gated ? 2 : 1) * out * a.row_bytes);
  const int64_t rows = groups * a.N * (gated ? 2 : 1);
  const bool mid = rows >= kRowsMid * static_cast<int64_t>(sms) && rows < kRowsLong * static_cast<int64_t>(sms);
  const int nw = type == DSQ_Q4_K && mid ? 12 : 8;
  // 8 warps: two slots each, about 140 KB in flight an SM, or four small ones; 12
  // warps: one, 110 KB; one too for Q8_0 pairs of the longest rows
  const size_t per_stage = static_cast<size_t>(nw) * a.slot_bytes;
  a.stages = per_stage <= 40 * 1024 ? 4 : per_stage <= 80 * 1024 ? 2 : 1;
  const size_t smem = per_stage * a.stages + nw * a.stages * sizeof(uint64_t);
  const RowsKernel kern = type == DSQ_Q8_0 ? rows_kernel<DSQ_Q8_0, 8>(G, gated, experts)
                          : nw == 8        ? rows_kernel<DSQ_Q4_K, 8>(G, gated, experts)
                                           : rows_kernel<DSQ_Q4_K, 12>(G, gated, experts);
  const int rc = set_smem_once(reinterpret_cast<const void *>(kern), static_cast<int>(smem), name);
  if (rc != DSQ_OK) return rc;
  const unsigned grid = static_cast<unsigned>(groups * a.per < sms ? groups * a.per : sms);
  const cudaError_t e = launch_pdl(kern, dim3(grid), dim3(nw * 32), smem, st, a);
  if (e != cudaSuccess) return fail(DSQ_ERR_LAUNCH, "%s: %s", name, cudaGetErrorString(e));
  return after_launch(name);
}

}  // namespace
}  // namespace dsq
