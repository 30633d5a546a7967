// gemv_fused.cu -- decode products with their epilogue, for prequantized tokens:
//   y[m][n] = act((W0 x_m)[n] + bias0[n]) [* ((W1 x_m)[n] + bias1[n])] + residual[m][n]
// for 1 to 8 tokens against one weight or a gate / up pair (dsq_gemv_fused),
// and for rows sorted by expert, each against its own expert's weights
// (dsq_gemv_experts).
//
// The sums are those of the multi-token GEMV (gemv_tokens.cu), term for term
// and in the same order, so without bias, activation and residual the outputs
// equal dsq_gemv_tokens bit for bit.
//
// HBM bound: every weight byte is read once per 8 tokens.  A row group is 32
// weight rows: 32 outputs of one weight, or 16 gate rows and the 16 up rows of
// the same outputs, so that both sums of an output end in one warp.  Each warp
// streams its units of a group (32 rows x 256 elements, 2-D TMA) through its own
// ring of shared-memory slots; the warps' partials meet in shared memory, and
// the warp that adds them up for a token applies the epilogue and stores.
// Where K has fewer units than the CTA has warps, the warps take several row
// groups side by side (an item); a CTA owns a contiguous run of items.
//
// Experts: the items are (tokens of one expert, row groups) in expert order,
// found on the device from the offsets of the sort, so nothing comes back to
// the host.  A CTA's run crosses few token groups, and while it exchanges the
// activations in shared memory the weight rings keep filling.
#include "epilogue.cuh"
#include "gemv_rows.cuh"
#include "tokens.cuh"

namespace dsq {
namespace {

constexpr int kFusedMaxE = 1024;

// Warps of a CTA.  One or two tokens: 16, which hide more of each other's
// latency (two tokens, N = 16384, K = 4096: Q8_0 17.5 us with 8, 14.7 with 16;
// Q4_K 17.0 and 12.5).  More tokens need the registers of 8: with 16 the
// tensor-core form measured slower (8 tokens Q8_0 19.1 -> 20.2 us, experts Q4_K
// 32.4 -> 38.1), except Q8_0 experts whose K has no more than 8 units, where two
// row groups run side by side (128 rows on 32 experts of 4096 x 2048: 69.9 -> 63.7).
int fused_warps(int type, int M, bool mma, bool experts, int G) {
  return M <= 2 || (mma && experts && type == DSQ_Q8_0 && G <= 8) ? 16 : 8;
}

struct FusedArgs {
  float *y;
  const float *bias[2];
  const float *residual;
  int act;
  int64_t N, K;
  int items;             // items of a weight (of one expert's): ceil(outputs / (side * group outputs))
  int nunits;            // K / 256
  int G;                 // virtual lanes per row (power of two, <= 32)
  int W;                 // warps on one row group: min(warps, G)
  int side;              // row groups of an item, side by side: at most warps / W
  int stages;            // ring slots per warp
  int M;                 // tokens (dsq_gemv_fused)
  uint32_t box_bytes, q_bytes, d_bytes, s_bytes, ring_off, bar_off, red_off;
  const int8_t *xq;
  const float *xd;
  const int32_t *xs;
  // experts
  const int32_t *offsets;   // [E + 1] first sorted row of each expert
  const int32_t *rows;      // [P] flat choice t*k + j of each sorted row, or NULL: row p reads activation p
  int E, k;
  int64_t P, A;             // sorted rows, activation rows
  WaitCtl wait;
};

// Where an item sits: token group c of expert e, item g of its weight.
struct ItemPos {
  int64_t item;
  int c, g, e;
};

// The expert tables of a CTA (E + 1 entries): first sorted row, first token
// group.
struct ExpertTables {
  int32_t off[kFusedMaxE + 1];
  int32_t group[kFusedMaxE + 1];
};

template <bool EXPERTS>
__device__ __forceinline__ ItemPos item_at(const FusedArgs &a, const ExpertTables *t, int64_t item) {
  ItemPos p{item, 0, static_cast<int>(item), 0};
  if constexpr (EXPERTS) {
    p.c = static_cast<int>(item / a.items);
    p.g = static_cast<int>(item - static_cast<int64_t>(p.c) * a.items);
    int lo = 0, hi = a.E;   // the last expert whose first group is <= c
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (t->group[mid] <= p.c) lo = mid;
      else hi = mid;
    }
    p.e = lo;
  }
  return p;
}

template <bool EXPERTS>
__device__ __forceinline__ void next_item(ItemPos &p, const FusedArgs &a, const ExpertTables *t) {
  ++p.item;
  ++p.g;
  if constexpr (EXPERTS) {
    if (p.g == a.items) {
      p.g = 0;
      ++p.c;
      while (p.e + 1 < a.E && t->group[p.e + 1] <= p.c) ++p.e;
    }
  }
}

// The virtual lanes of a warp are taken in the order their sums meet: with four
// of them (0 + 2) + (1 + 3), with two 0 + 1.
__device__ __forceinline__ int lane_slot(int step, int vpw) { return vpw == 4 ? ((step & 1) << 1) | (step >> 1) : step; }

// A warp's boxes in the order it consumes them: item, virtual lane (step i), unit
// u.  w: the warp's number within its row group.
template <bool EXPERTS>
struct BoxCursor {
  ItemPos p;
  int64_t end;
  int i, u;
  __device__ __forceinline__ void first(const FusedArgs &a, const ItemPos &from, int64_t hi, int w, int vpw) {
    p = from;
    end = (vpw == 0 || w >= a.nunits) ? p.item : hi;   // no units for this warp: no boxes
    i = 0;
    u = w;
  }
  __device__ __forceinline__ bool valid() const { return p.item < end; }
  __device__ __forceinline__ void next(const FusedArgs &a, const ExpertTables *t, int w, int vpw) {
    u += a.G;
    if (u < a.nunits) return;
    while (++i < vpw) {
      u = w + a.W * lane_slot(i, vpw);
      if (u < a.nunits) return;
    }
    i = 0;
    u = w;
    next_item<EXPERTS>(p, a, t);
  }
  // first weight row of the box (of each box of a pair)
  template <int OUT>
  __device__ __forceinline__ int32_t row0(const FusedArgs &a, int sub) const {
    return static_cast<int32_t>((EXPERTS ? p.e * a.N : 0) + (static_cast<int64_t>(p.g) * a.side + sub) * OUT);
  }
};

// Activation row of sorted row p, -1 outside the activations.
__device__ __forceinline__ int64_t source_row(const FusedArgs &a, int64_t p) {
  int64_t r = p;
  if (a.rows) {
    const int32_t f = a.rows[p];
    r = f < 0 ? -1 : f / a.k;
  }
  return r < a.A ? r : -1;
}

template <int TYPE, int M, bool MMA, bool EXPERTS, bool GATED, int NW>
__global__ void __launch_bounds__(NW * 32, 1)
    gemv_fused_kernel(const __grid_constant__ CUtensorMap map0, const __grid_constant__ CUtensorMap map1,
                      const __grid_constant__ FusedArgs a) {
  constexpr int UB = tok_unit_bytes<TYPE>();
  constexpr int NT = NW * 32;
  constexpr int NA = MMA ? 8 : M;   // sums a lane holds
  constexpr int VL = 32 / NW;       // most virtual lanes of a warp
  constexpr int OUT = GATED ? kTokRows / 2 : kTokRows;   // outputs of a row group
  extern __shared__ uint8_t smem_raw[];
  uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  ExpertTables *tables = nullptr;
  if constexpr (EXPERTS) {
    __shared__ ExpertTables shared_tables;
    tables = &shared_tables;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int grp = lane >> 2, t = lane & 3;
  const int W = a.W, S = a.stages;
  const int sub = warp / W, w = warp - sub * W;   // this warp's row group of the item, its number there
  const int vpw = sub < a.side ? a.G / W : 0;     // its virtual lanes
  uint8_t *act_q = base;
  float *act_d = reinterpret_cast<float *>(base + a.q_bytes);
  int32_t *act_s = reinterpret_cast<int32_t *>(base + a.q_bytes + a.d_bytes);
  uint8_t *ring = base + a.ring_off + static_cast<size_t>(warp) * S * a.box_bytes;
  uint64_t *bars = reinterpret_cast<uint64_t *>(base + a.bar_off) + warp * kTokMaxStages;
  uint64_t *act_bar = reinterpret_cast<uint64_t *>(base + a.bar_off) + NW * kTokMaxStages + 1;
  float *red = reinterpret_cast<float *>(base + a.red_off);   // [2][warps][M][32 rows]
  volatile uint32_t *abort_flag =
      reinterpret_cast<volatile uint32_t *>(reinterpret_cast<uint64_t *>(base + a.bar_off) + NW * kTokMaxStages);

  if (threadIdx.x == 0) {
    *abort_flag = 0u;
    mbar_init(act_bar, 1);
    prefetch_tensormap(&map0);
    if (GATED) prefetch_tensormap(&map1);
  }
  if (lane == 0)
    for (int s = 0; s < S; ++s) mbar_init(&bars[s], 1);
  fence_barrier_init();
  int64_t items = a.items, lo, hi;
  // this CTA's items: as even a share as there is (32-bit where it fits)
  auto share = [&]() {
    if (items < (int64_t(1) << 20)) {
      const uint32_t n = static_cast<uint32_t>(items), each = n / gridDim.x, more = n - each * gridDim.x;
      lo = each * blockIdx.x + min(blockIdx.x, more);
      hi = lo + each + (blockIdx.x < more ? 1 : 0);
    } else {
      lo = items * blockIdx.x / gridDim.x;
      hi = items * (blockIdx.x + 1) / gridDim.x;
    }
  };
  ItemPos p{};
  BoxCursor<EXPERTS> issue;
  if constexpr (!EXPERTS) {
    // weights are read-only: bring this warp's first boxes toward L2 while
    // the kernel before us finishes
    share();
    p = item_at<EXPERTS>(a, tables, lo);
    issue.first(a, p, hi, w, vpw);
    if (lane == 0) {
      BoxCursor<EXPERTS> c = issue;
      for (int s = 0; s < S && c.valid(); ++s, c.next(a, tables, w, vpw)) {
        prefetch_l2_tile_2d(&map0, c.u * (UB / 4), c.template row0<OUT>(a, sub));
        if (GATED) prefetch_l2_tile_2d(&map1, c.u * (UB / 4), c.template row0<OUT>(a, sub));
      }
    }
  }
  __syncthreads();
  pdl_trigger();
  pdl_wait();
  if constexpr (EXPERTS) {
    // offsets, clamped to the rows there are, and the token groups of each expert
    for (int e = threadIdx.x; e <= a.E; e += NT)
      tables->off[e] = static_cast<int32_t>(min(max(static_cast<int64_t>(a.offsets[e]), int64_t(0)), a.P));
    __syncthreads();
    if (warp == 0) {
      const int per = (a.E + 31) / 32;
      const int e0 = min(lane * per, a.E), e1 = min(e0 + per, a.E);
      // offsets that fall back are lifted to the largest before them, so that
      // whatever they hold the groups are within the rows there are
      int32_t top = 0;
      for (int e = e0; e < e1; ++e) top = max(top, tables->off[e]);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int32_t up = __shfl_up_sync(0xffffffffu, top, o);
        if (lane >= o) top = max(top, up);
      }
      int32_t before = __shfl_up_sync(0xffffffffu, top, 1);
      if (lane == 0) before = 0;
      for (int e = e0; e < e1; ++e) tables->off[e] = before = max(before, tables->off[e]);
      if (lane == 31) tables->off[a.E] = max(top, tables->off[a.E]);
      __syncwarp();
      int32_t sum = 0;
      for (int e = e0; e < e1; ++e) sum += (tables->off[e + 1] - tables->off[e] + M - 1) / M;
      int32_t inc = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int32_t up = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += up;
      }
      int32_t at = inc - sum;
      for (int e = e0; e < e1; ++e) {
        tables->group[e] = at;
        at += (tables->off[e + 1] - tables->off[e] + M - 1) / M;
      }
      if (lane == 31) tables->group[a.E] = at;
    }
    __syncthreads();
    items = static_cast<int64_t>(tables->group[a.E]) * a.items;
    share();
    p.item = lo;
    if (lo < hi) p = item_at<EXPERTS>(a, tables, lo);
    issue.first(a, p, hi, w, vpw);
  }

  uint32_t act_parity = 0;
  int cnt = a.M;         // tokens of the group at hand
  int64_t row_out = 0;   // its first output row
  // Where the tokens of position p's group sit.
  auto enter_group = [&]() {
    if constexpr (EXPERTS) {
      row_out = tables->off[p.e] + static_cast<int64_t>(p.c - tables->group[p.e]) * M;
      cnt = static_cast<int>(min(static_cast<int64_t>(M), tables->off[p.e + 1] - row_out));
    }
  };
  // Starts the group's activations towards shared memory: bulk copies of the
  // [token] rows of codes, scales and sums (contiguous rows of a call, or one
  // expert row).  The tensor-core form lays them out itself.
  auto start_act = [&]() {
    if constexpr (!MMA) {
      const int64_t src = EXPERTS ? source_row(a, row_out) : 0;
      if (src >= 0) {
        const uint64_t keep = l2_policy_evict_last();
        mbar_arrive_expect_tx(act_bar, a.q_bytes + a.d_bytes + a.s_bytes);
        bulk_g2s(act_q, a.xq + src * a.K, a.q_bytes, act_bar, keep);
        bulk_g2s(act_d, a.xd + src * (a.K / 32), a.d_bytes, act_bar, keep);
        if (TYPE == DSQ_Q4_K) bulk_g2s(act_s, a.xs + src * (a.K / 32), a.s_bytes, act_bar, keep);
      }
    }
  };
  bool started = false;   // the first group's copies are under way
  if (lo < hi) {
    enter_group();
    if (threadIdx.x == 0) start_act();
    started = true;
  }
  int64_t n_issued = 0, n_waited = 0;
  auto issue_box = [&](int slot) {
    uint8_t *dst = ring + static_cast<size_t>(slot) * a.box_bytes;
    const int32_t row0 = issue.template row0<OUT>(a, sub);
    mbar_arrive_expect_tx(&bars[slot], a.box_bytes);
    tma_load_2d(dst, &map0, issue.u * (UB / 4), row0, &bars[slot]);
    if (GATED) tma_load_2d(dst + OUT * UB, &map1, issue.u * (UB / 4), row0, &bars[slot]);
    issue.next(a, tables, w, vpw);
    ++n_issued;
  };
  if (lane == 0)
    for (int s = 0; s < S && issue.valid(); ++s) issue_box(s);

  bool ok = true;
  int slot = 0;
  uint32_t parity = 0;
  int buf = 0;
  int have = -1;   // token group whose activations are in shared memory
  for (; p.item < hi; next_item<EXPERTS>(p, a, tables), buf ^= 1) {
    if (p.c != have) {
      if (have >= 0) __syncthreads();   // every warp is done with the activations it replaces
      have = p.c;
      if (!started) {
        enter_group();
        if (threadIdx.x == 0) {
          fence_proxy_async_smem();   // after the reads of what the copies replace
          start_act();
        }
      }
      started = false;
      if constexpr (MMA) {
        // [unit][block][chunk][8 tokens] words, tokens past cnt zero (plain loads:
        // the kernel before writes them, and read-only loads may pass the wait for it)
        const uint32_t words = static_cast<uint32_t>(a.K / 4), nb = static_cast<uint32_t>(a.K / 32);
        int64_t src[8];
#pragma unroll
        for (int tok = 0; tok < 8; ++tok)
          src[tok] = tok < cnt ? (EXPERTS ? source_row(a, row_out + tok) : tok) : -1;
        const uint32_t *xq32 = reinterpret_cast<const uint32_t *>(a.xq);
        constexpr int kAhead = 4;   // words a thread has under way for each token
        for (uint32_t w0 = threadIdx.x; w0 < words; w0 += kAhead * NT) {
          uint32_t v[kAhead][8];
#pragma unroll
          for (int j = 0; j < kAhead; ++j)
#pragma unroll
            for (int tok = 0; tok < 8; ++tok)
              v[j][tok] = src[tok] >= 0 && w0 + j * NT < words ? xq32[src[tok] * words + w0 + j * NT] : 0u;
#pragma unroll
          for (int j = 0; j < kAhead; ++j) {
            if (w0 + j * NT >= words) break;
            uint4 *dst = reinterpret_cast<uint4 *>(act_q) + act_chunk(w0 + j * NT) * 2;
            dst[0] = make_uint4(v[j][0], v[j][1], v[j][2], v[j][3]);
            dst[1] = make_uint4(v[j][4], v[j][5], v[j][6], v[j][7]);
          }
        }
        for (uint32_t blk = threadIdx.x; blk < nb; blk += NT) {
          float d[8];
          float sm[8];
#pragma unroll
          for (int tok = 0; tok < 8; ++tok) {
            d[tok] = src[tok] >= 0 ? a.xd[src[tok] * nb + blk] : 0.0f;
            sm[tok] = (TYPE == DSQ_Q4_K && src[tok] >= 0) ? static_cast<float>(a.xs[src[tok] * nb + blk]) : 0.0f;
          }
          float4 *dd = reinterpret_cast<float4 *>(act_d) + blk * 2;
          dd[0] = make_float4(d[0], d[1], d[2], d[3]);
          dd[1] = make_float4(d[4], d[5], d[6], d[7]);
          if (TYPE == DSQ_Q4_K) {
            float4 *ds = reinterpret_cast<float4 *>(act_s) + blk * 2;
            ds[0] = make_float4(sm[0], sm[1], sm[2], sm[3]);
            ds[1] = make_float4(sm[4], sm[5], sm[6], sm[7]);
          }
        }
        __syncthreads();
      } else if (!EXPERTS || source_row(a, row_out) >= 0) {
        const bool got = mbar_wait_for(act_bar, act_parity, a.wait.limit_ns);
        act_parity ^= 1u;
        if (!__all_sync(0xffffffffu, got)) {
          ok = false;
          if (lane == 0 && *abort_flag == 0u) {
            *abort_flag = 1u;
            record_timeout(a.wait);
          }
          // the copies still in flight land before the area is used again
          mbar_wait_for(act_bar, act_parity ^ 1u, kDrainLimitNs);
        }
      } else {
        const uint32_t words = (a.q_bytes + a.d_bytes + a.s_bytes) / 16;
        for (uint32_t wd = threadIdx.x; wd < words; wd += NT)
          reinterpret_cast<uint4 *>(act_q)[wd] = make_uint4(0u, 0u, 0u, 0u);
        __syncthreads();
      }
    }
    // what the warp's first task adds, under way before the units are waited for
    float pre_bias = 0.0f, pre_res = 0.0f;
    if (warp < a.side * M && warp % M < cnt) {
      const int64_t n = (static_cast<int64_t>(p.g) * a.side + warp / M) * OUT + (GATED ? lane & 15 : lane);
      const float *bias = a.bias[GATED ? lane >> 4 : 0];
      if (n < a.N) {
        if (bias) pre_bias = bias[(EXPERTS ? p.e * a.N : 0) + n];
        if (a.residual && (!GATED || lane < 16)) pre_res = a.residual[(row_out + warp % M) * a.N + n];
      }
    }
    // one copy of the unit's code, whatever the number of virtual lanes: copies
    // evicted each other from the instruction cache (a unit took 2400 cycles in
    // a fresh copy, 1130 in a warm one)
    float cur[NA], held[VL == 4 ? NA : 1];
    for (int i = 0; i < vpw; ++i) {
      float acc[NA];
#pragma unroll
      for (int v = 0; v < NA; ++v) acc[v] = 0.0f;
      for (int u = w + W * lane_slot(i, vpw); u < a.nunits; u += a.G) {
        if (ok) {
          bool got = a.wait.limit_ns > 0 && mbar_try_wait(&bars[slot], parity);
          if (!got) got = *abort_flag == 0u && mbar_wait_for(&bars[slot], parity, a.wait.limit_ns);
          ok = __all_sync(0xffffffffu, got);
          if (!ok && lane == 0 && *abort_flag == 0u) {
            *abort_flag = 1u;
            record_timeout(a.wait);
          }
        }
        if (ok) {
          ++n_waited;
          float part[NA];
          const uint8_t *box = ring + static_cast<size_t>(slot) * a.box_bytes;
          if constexpr (MMA) {
            const uint32_t *q32 = reinterpret_cast<const uint32_t *>(act_q);
            if constexpr (TYPE == DSQ_Q8_0)
              tok_pair_q8_0(box, q32, act_d, u, lane, part);
            else
              tok_pair_q4_k(box, q32, act_d, reinterpret_cast<const float *>(act_s), u, lane, part);
          } else {
            const uint8_t *rowp = box + static_cast<size_t>(lane) * UB;
            const int8_t *q8 = reinterpret_cast<const int8_t *>(act_q);
            if constexpr (TYPE == DSQ_Q8_0)
              tok_unit_q8_0<M>(rowp, q8, act_d, a.K, u, part, nullptr, 0);
            else
              tok_unit_q4_k<M>(rowp, q8, act_d, act_s, a.K, u, part, nullptr, 0);
          }
#pragma unroll
          for (int v = 0; v < NA; ++v) acc[v] += part[v];
          __syncwarp();
          if (lane == 0 && issue.valid()) {
            fence_proxy_async_smem();
            issue_box(slot);
          }
        }
        if (++slot == S) {
          slot = 0;
          parity ^= 1u;
        }
      }
      // butterfly strides >= W stay inside the warp (gemv_tokens.cu)
#pragma unroll
      for (int v = 0; v < NA; ++v) {
        if (i == 0) {
          cur[v] = acc[v];
        } else if (VL == 4 && i == 2) {
          held[VL == 4 ? v : 0] = cur[v];
          cur[v] = acc[v];
        } else {
          cur[v] += acc[v];
        }
        if (VL == 4 && i == 3) cur[v] = held[VL == 4 ? v : 0] + cur[v];
      }
    }
    // ... the rest cross warps, the largest stride first
    float *rb = red + static_cast<size_t>(buf) * NW * M * 32;
    if (vpw > 0) {
#pragma unroll
      for (int v = 0; v < NA; ++v) {
        if constexpr (MMA) rb[(warp * M + mma_tok(v, t)) * 32 + mma_row(v, grp)] = cur[v];
        else rb[(warp * M + v) * 32 + lane] = cur[v];
      }
    }
    __syncthreads();
    for (int task = warp; task < a.side * M; task += NW) {   // a token of a row group
      const int tok = task % M, side = task / M;
      if (tok >= cnt) continue;
      const float *rs = rb + (side * W * M + tok) * 32 + lane;
      float r[NW];
#pragma unroll
      for (int j = 0; j < NW; ++j) r[j] = j < W ? rs[j * M * 32] : 0.0f;
#pragma unroll
      for (int o = NW / 2; o >= 1; o >>= 1)
        if (o < W) {
#pragma unroll
          for (int j = 0; j < o; ++j) r[j] += r[j + o];
        }
      const int64_t n = (static_cast<int64_t>(p.g) * a.side + side) * OUT + (GATED ? lane & 15 : lane);
      float v = r[0];
      const float *bias = a.bias[GATED ? lane >> 4 : 0];
      if (bias && n < a.N) v = __fadd_rn(v, task == warp ? pre_bias : bias[(EXPERTS ? p.e * a.N : 0) + n]);
      const float up = GATED ? __shfl_down_sync(0xffffffffu, v, 16) : 0.0f;
      if (n < a.N && (!GATED || lane < 16) && *abort_flag == 0u) {
        v = activate(v, a.act);
        if (GATED) v = __fmul_rn(v, up);
        const int64_t at = (row_out + tok) * a.N + n;
        if (a.residual) v = __fadd_rn(v, task == warp ? pre_res : a.residual[at]);
        a.y[at] = v;
      }
    }
  }
  // after an abort: let this warp's copies still in flight land before exit
  if (lane == 0)
    for (int64_t j = n_waited; j < n_issued; ++j)
      mbar_wait_for(&bars[j % S], static_cast<uint32_t>((j / S) & 1), kDrainLimitNs);
}

using FusedKernel = void (*)(const CUtensorMap, const CUtensorMap, const FusedArgs);

// The kernel for M tokens per group; experts take groups of 1 or 8.
template <int TYPE, bool EXPERTS, bool GATED>
FusedKernel fused_kernel(int M, bool mma, [[maybe_unused]] int nw) {
  if constexpr (EXPERTS && TYPE == DSQ_Q8_0)
    if (mma && nw == 16) return gemv_fused_kernel<TYPE, 8, true, true, GATED, 16>;
  if (mma) return gemv_fused_kernel<TYPE, 8, true, EXPERTS, GATED, 8>;
  if constexpr (EXPERTS) {
    return gemv_fused_kernel<TYPE, 1, false, true, GATED, 16>;
  } else {
    switch (M) {
      case 1: return gemv_fused_kernel<TYPE, 1, false, false, GATED, 16>;
      case 2: return gemv_fused_kernel<TYPE, 2, false, false, GATED, 16>;
      case 3: return gemv_fused_kernel<TYPE, 3, false, false, GATED, 8>;
      case 4: return gemv_fused_kernel<TYPE, 4, false, false, GATED, 8>;
      case 5: return gemv_fused_kernel<TYPE, 5, false, false, GATED, 8>;
      case 6: return gemv_fused_kernel<TYPE, 6, false, false, GATED, 8>;
      default: return gemv_fused_kernel<TYPE, 7, false, false, GATED, 8>;   // 8 that fit take the tensor cores
    }
  }
}

size_t act_bytes_per_token(int type, int64_t K) {
  return static_cast<size_t>(K) + (K / 32) * 4 * (type == DSQ_Q4_K ? 2 : 1);
}

// Launches the kernel for `a` with M tokens per group (the rest of `a` that
// depends on the shape is filled in here).  groups: token groups there can be.
template <int TYPE, bool EXPERTS>
int fused_launch(const char *name, FusedArgs &a, int M, bool mma, const void *w0, const void *w1, int64_t rows,
                 int64_t groups, int sms, cudaStream_t st) {
  const int64_t K = a.K;
  const int out = w1 ? kTokRows / 2 : kTokRows;
  a.nunits = static_cast<int>(K / 256);
  a.G = 1;
  while (a.G < a.nunits && a.G < 32) a.G <<= 1;
  const int nw = fused_warps(TYPE, M, mma, EXPERTS, a.G);
  a.W = a.G < nw ? a.G : nw;
  // row groups side by side: as many as the warps have room for, as long as
  // every SM still gets an item
  const int64_t row_groups = (a.N + out - 1) / out;
  a.side = 1;
  while (2 * a.side * a.W <= nw && groups * row_groups >= 2 * a.side * static_cast<int64_t>(sms)) a.side *= 2;
  a.items = static_cast<int>((row_groups + a.side - 1) / a.side);
  a.box_bytes = static_cast<uint32_t>(kTokRows * (TYPE == DSQ_Q8_0 ? 272 : 144));
  a.q_bytes = static_cast<uint32_t>(M * K);
  a.d_bytes = static_cast<uint32_t>(M * (K / 32) * 4);
  a.s_bytes = TYPE == DSQ_Q4_K ? a.d_bytes : 0;
  // shared memory: activations | ring (warps x stages x box) | barriers |
  // reduction
  const size_t act = tok_align(a.q_bytes + a.d_bytes + a.s_bytes, 1024);
  const size_t bars = tok_align((nw * kTokMaxStages + 2) * sizeof(uint64_t), 16);
  const size_t red = 2 * static_cast<size_t>(nw) * M * 32 * sizeof(float);
  const size_t fixed = 1024 + act + bars + red + (EXPERTS ? sizeof(ExpertTables) : 0);
  const size_t per_stage = static_cast<size_t>(nw) * a.box_bytes;
  int stages = fixed < kTokSmemLimit ? static_cast<int>((kTokSmemLimit - fixed) / per_stage) : 0;
  if (stages > kTokMaxStages) stages = kTokMaxStages;
  DSQ_REQUIRE(stages >= 1, DSQ_ERR_SHAPE, "%s: no pipeline fits next to the activations of K=%lld", name,
              (long long)K);
  a.stages = stages;
  a.ring_off = static_cast<uint32_t>(act);
  a.bar_off = static_cast<uint32_t>(act + per_stage * stages);
  a.red_off = static_cast<uint32_t>(a.bar_off + bars);
  const size_t smem = 1024 + a.red_off + red;
  CUtensorMap m0, m1;
  int rc = tok_map(&m0, w0, TYPE, rows, K, name, out);
  if (rc != DSQ_OK) return rc;
  m1 = m0;
  if (w1) {
    rc = tok_map(&m1, w1, TYPE, rows, K, name, out);
    if (rc != DSQ_OK) return rc;
  }
  const FusedKernel kern = w1 ? fused_kernel<TYPE, EXPERTS, true>(M, mma, nw)
                              : fused_kernel<TYPE, EXPERTS, false>(M, mma, nw);
  rc = set_smem_once(reinterpret_cast<const void *>(kern), static_cast<int>(smem), name);
  if (rc != DSQ_OK) return rc;
  const int64_t most = groups * a.items;
  const unsigned grid = static_cast<unsigned>(most < sms ? most : sms);
  const cudaError_t e = launch_pdl(kern, dim3(grid), dim3(nw * 32), smem, st, m0, m1, a);
  if (e != cudaSuccess) return fail(DSQ_ERR_LAUNCH, "%s: %s", name, cudaGetErrorString(e));
  return after_launch(name);
}

RowsArgs rows_args(const FusedArgs &f, const void *w0, const void *w1) {
  RowsArgs a{};
  a.w[0] = static_cast<const uint8_t *>(w0);
  a.w[1] = static_cast<const uint8_t *>(w1);
  a.y = f.y;
  a.bias[0] = f.bias[0];
  a.bias[1] = f.bias[1];
  a.residual = f.residual;
  a.act = f.act;
  a.N = f.N;
  a.K = f.K;
  a.xq = f.xq;
  a.xd = f.xd;
  a.xs = f.xs;
  a.offsets = f.offsets;
  a.rows = f.rows;
  a.E = f.E;
  a.k = f.k;
  a.P = static_cast<int>(f.P);
  a.A = f.A;
  a.wait = f.wait;
  return a;
}

// One token by rows or by boxes (rows: weight rows of the call; K = 4096, one
// weight).  Rows win on short matrices (1024 rows: 2.8 against 3.5 us), which
// leave most SMs without a box, and on long ones (16384 rows: Q8_0 11.7 against
// 12.7, Q4_K 10.3 against 11.8); between 2048 rows and one row group per SM the
// boxes spread one row over 16 warps (4096 rows Q4_K: 4.1 against 4.6).
bool one_token_by_rows(int64_t rows, int sms) { return rows < 2048 || rows > 32 * static_cast<int64_t>(sms); }

// The checks both entry points share.
int fused_validate(const char *name, int type, const void *w0, const void *w1, int64_t N, int64_t K, const int8_t *xq,
                   const float *xd, const int32_t *xs, int act, const float *bias0, const float *bias1,
                   const float *y) {
  DSQ_REQUIRE(type == DSQ_Q8_0 || type == DSQ_Q4_K, DSQ_ERR_INVALID_ARG, "%s: unsupported type %d", name, type);
  DSQ_REQUIRE(K > 0 && N >= 0, DSQ_ERR_INVALID_ARG, "%s: N=%lld K=%lld", name, (long long)N, (long long)K);
  DSQ_REQUIRE(valid_act(act), DSQ_ERR_INVALID_ARG, "%s: unknown activation %d", name, act);
  DSQ_REQUIRE(w1 || !bias1, DSQ_ERR_INVALID_ARG, "%s: bias1 needs a second weight", name);
  DSQ_REQUIRE(K % 256 == 0, DSQ_ERR_SHAPE, "%s: K=%lld must be a multiple of 256", name, (long long)K);
  DSQ_REQUIRE(N <= (int64_t(1) << 30), DSQ_ERR_SHAPE, "%s: too many rows", name);
  DSQ_REQUIRE(act_bytes_per_token(type, K) <= kTokMaxActSmem, DSQ_ERR_SHAPE,
              "%s: a token of K=%lld exceeds the %zu bytes of shared memory kept for activations", name, (long long)K,
              kTokMaxActSmem);
  if (N == 0) return DSQ_OK;
  DSQ_REQUIRE(xq && xd && (type == DSQ_Q8_0 || xs), DSQ_ERR_INVALID_ARG, "%s: null activation pointer", name);
  DSQ_REQUIRE(w0 && y, DSQ_ERR_INVALID_ARG, "%s: null weight/output pointer", name);
  DSQ_REQUIRE(aligned(xq, 16) && aligned(xd, 16) && (type == DSQ_Q8_0 || aligned(xs, 16)), DSQ_ERR_ALIGNMENT,
              "%s: xq/xd/xs must be 16-byte aligned", name);
  DSQ_REQUIRE(aligned(w0, 16) && aligned(w1, 16) && aligned(y, 4) && aligned(bias0, 4) && aligned(bias1, 4),
              DSQ_ERR_ALIGNMENT, "%s: weights must be 16-byte, biases and outputs 4-byte aligned", name);
  return DSQ_OK;
}

}  // namespace
}  // namespace dsq

extern "C" int dsq_gemv_fused(int type, const void *w0, const void *w1, int64_t N, int64_t K, int64_t M,
                              const int8_t *xq, const float *xd, const int32_t *xs, int act, const float *bias0,
                              const float *bias1, const float *residual, float *y, void *stream) {
  using namespace dsq;
  const char *name = "dsq_gemv_fused";
  DSQ_REQUIRE(M >= 1 && M <= kTokMaxM, DSQ_ERR_SHAPE, "%s: M=%lld tokens (1..%d supported)", name, (long long)M,
              kTokMaxM);
  int rc = fused_validate(name, type, w0, w1, N, K, xq, xd, xs, act, bias0, bias1, y);
  if (rc != DSQ_OK) return rc;
  DSQ_REQUIRE(aligned(residual, 4), DSQ_ERR_ALIGNMENT, "%s: residual must be 4-byte aligned", name);
  const size_t per_token = act_bytes_per_token(type, K);
  DSQ_REQUIRE(M * per_token <= kTokMaxActSmem, DSQ_ERR_SHAPE,
              "%s: %lld tokens of K=%lld exceed the %zu bytes of shared memory kept for activations", name,
              (long long)M, (long long)K, kTokMaxActSmem);
  if (N == 0) return DSQ_OK;
  FusedArgs a{};
  int sms = 0;
  rc = wait_ctl(&a.wait, &sms);
  if (rc != DSQ_OK) return rc;
  a.y = y;
  a.bias[0] = bias0;
  a.bias[1] = bias1;
  a.residual = residual;
  a.act = act;
  a.N = N;
  a.K = K;
  a.M = static_cast<int>(M);
  a.xq = xq;
  a.xd = xd;
  a.xs = xs;
  cudaStream_t st = as_stream(stream);
  if (M == 1 && rows_fit(K, N, 1) && one_token_by_rows(w1 ? 2 * N : N, sms)) {
    RowsArgs r = rows_args(a, w0, w1);
    return rows_launch(name, type, r, w1 != nullptr, false, 1, sms, st);
  }
  // the tensor cores from the token count gemv_tokens.cu takes them from
  const bool mma = M >= tok_mma_min_m(type) && 8 * per_token <= kTokMaxActSmem;
  const int Mk = mma ? 8 : a.M;
  return type == DSQ_Q8_0 ? fused_launch<DSQ_Q8_0, false>(name, a, Mk, mma, w0, w1, N, 1, sms, st)
                          : fused_launch<DSQ_Q4_K, false>(name, a, Mk, mma, w0, w1, N, 1, sms, st);
}

extern "C" int dsq_gemv_experts(int type, const void *w0, const void *w1, int64_t E, int64_t N, int64_t K,
                                const int32_t *offsets, const int32_t *rows, int64_t k, int64_t P, const int8_t *xq,
                                const float *xd, const int32_t *xs, int64_t A, int act, const float *bias0,
                                const float *bias1, float *y, void *stream) {
  using namespace dsq;
  const char *name = "dsq_gemv_experts";
  DSQ_REQUIRE(E >= 1 && P >= 0 && A >= 0 && k >= 1, DSQ_ERR_INVALID_ARG, "%s: E=%lld P=%lld A=%lld k=%lld", name,
              (long long)E, (long long)P, (long long)A, (long long)k);
  DSQ_REQUIRE(E <= kFusedMaxE && P <= (int64_t(1) << 30) && A <= (int64_t(1) << 30) && k <= (int64_t(1) << 30),
              DSQ_ERR_SHAPE, "%s: size out of range (E <= %d, P and A <= 2^30)", name, kFusedMaxE);
  int rc = fused_validate(name, type, w0, w1, N, K, xq, xd, xs, act, bias0, bias1, y);
  if (rc != DSQ_OK) return rc;
  DSQ_REQUIRE(E * N < (int64_t(1) << 31) - 32, DSQ_ERR_SHAPE, "%s: the experts hold more than 2^31 rows", name);
  if (N == 0 || P == 0) return DSQ_OK;
  DSQ_REQUIRE(offsets != nullptr, DSQ_ERR_INVALID_ARG, "%s: null offsets", name);
  DSQ_REQUIRE(aligned(offsets, 4) && aligned(rows, 4), DSQ_ERR_ALIGNMENT, "%s: offsets and rows must be 4-byte aligned",
              name);
  FusedArgs a{};
  int sms = 0;
  rc = wait_ctl(&a.wait, &sms);
  if (rc != DSQ_OK) return rc;
  a.y = y;
  a.bias[0] = bias0;
  a.bias[1] = bias1;
  a.act = act;
  a.N = N;
  a.K = K;
  a.M = 1;
  a.xq = xq;
  a.xd = xd;
  a.xs = xs;
  a.offsets = offsets;
  a.rows = rows;
  a.E = static_cast<int>(E);
  a.k = static_cast<int>(k);
  a.P = P;
  a.A = A;
  // One sorted row at a time streams a weight once per row, fastest while an
  // expert has about one; groups of 8 read it once for all its rows, but the
  // tensor-core form unpacks at 1.5 (Q8_0) to 3 (Q4_K) times the memory's pace.
  // 32 experts of 4096 x 2048, tokens that choose 4 of them at random, one row /
  // groups: Q8_0 30 / 36 us at 24 rows, 39 / 40 at 28, 45 / 39 at 32, 79 / 54 at 64;
  // Q4_K 29 / 41 at 32, 49 / 60 at 64, 88 / 70 at 128.  Uneven choices (by 1 / rank)
  // favour the groups a little sooner, 35 / 32 at 28 rows of Q8_0; rows spread
  // evenly, a program's exception, favour single rows longer, 46 / 58 at 32.
  const bool mma = 4 * P > (type == DSQ_Q8_0 ? 3 : 8) * E && 8 * act_bytes_per_token(type, K) <= kTokMaxActSmem;
  cudaStream_t st = as_stream(stream);
  if (!mma && rows_fit(K, N, P)) {
    RowsArgs r = rows_args(a, w0, w1);
    return rows_launch(name, type, r, w1 != nullptr, true, P, sms, st);
  }
  return type == DSQ_Q8_0 ? fused_launch<DSQ_Q8_0, true>(name, a, mma ? 8 : 1, mma, w0, w1, E * N, P, sms, st)
                          : fused_launch<DSQ_Q4_K, true>(name, a, mma ? 8 : 1, mma, w0, w1, E * N, P, sms, st);
}
