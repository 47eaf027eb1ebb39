// The whole MoE layer for a few tokens (1 .. 16) in two launches.
//
//   l_t = x_t W_g (+ b_g);  (e_tj, p_tj) = top-k of l_t, softmax over the kept
//   h_te = p_tj * silu(x_t W1_e^T) * (x_t W3_e^T)         for kept (t, j), e = e_tj
//   y_t  = sum_e h_te W2_e^T  (+ the shared expert, weight 1 or 1 + dropped)
//
// What bounds it: the touched experts' weights, read once from HBM; next to
// them everything else (x, h, the router) is small and comes from L2.  The
// general path spends 6 to 9 launches and row tiles of 32 to 256 rows on it.
//
//   few_router_kernel  split-K partial logits, and zeroes the counters
//   few_layer_kernel   everything else.  Every workgroup selects and groups the
//                      few tokens for itself (no wait), then takes work items from
//                      a queue in ticket order: gate/up tiles segment by segment
//                      (a segment is one touched expert), then down tiles.  A
//                      down item waits until its segments' gate/up tiles are done;
//                      these all have lower tickets, so they are held by
//                      workgroups that already run, and gate/up items wait for
//                      nothing.  Every wait therefore ends however few workgroups
//                      the device runs at once, whatever else runs on it.
//
// With at most 16 tokens the MFMA's 16 columns are the tokens themselves: no
// gather, no permutation; a token without the segment's expert is a column of
// zeros (its loads are sent out of range, which costs no traffic).  A workgroup
// is eight waves, one workgroup per CU, that share an item's rows and split its k
// range; their partial tiles are summed through LDS in wave order.  The routing weight is folded
// into h, h is kept in three bf16 terms (24 bits: as exact as fp32, and bf16
// MFMA time is free here), and the k pieces of a row of y are added in order,
// so results do not depend on timing: equal calls give equal bits.
//
// Loop control is scalar throughout: tickets, segments, steps and what waits compare
// pass through uniform() wherever they come from LDS or memory, and no loop that lanes
// leave one by one keeps values alive that are used after it.  This is not for speed.
// A form with such values in vector registers was compiled with the copy of a live
// one placed at the end of a divergent loop, where the execution mask is still empty:
// the copy wrote nothing, the item count came back as what the register had held, and
// tickets past the last item were worked on at addresses out of range.
#include <algorithm>

#include "moe_internal.h"
#include "topk_key.h"
#include "weight_stream.h"

namespace moe {
namespace {

constexpr int kWaves = 8;             // waves of a workgroup
constexpr int kThreads = kWaves * 64;
constexpr int kCols = kFewColumns;    // tokens of a call at most
// Output rows of a down item (the last may have 64 of 128).  Eight row tiles share
// each load of h: with four, the loads of its three terms cost as much as narrow
// weights' (16 tokens, int4, Mixtral widths: 266 us against 251); bf16 weights are
// twice the bytes or more and gain from the finer split over workgroups (one token:
// 148 us against 152, of 64 experts 33 against 36).
constexpr int kDownRowsMin = 64;
constexpr int down_rows(int wq) { return wq == WS_BF16 ? kDownRowsMin : 128; }
constexpr int kMaxSplits = 8;         // K splits of the router at most
constexpr int kMaxPieces = 16;        // k pieces the down items of a row tile are cut into

struct FewParams {
  const uint16_t* x;      // [T, d]
  const float* partial;   // [T, splits, E]
  const float* b_g;
  const void* W1; const void* W3; const void* W2;
  const float* s1; const float* s3; const float* s2;
  const void* W1s; const void* W3s; const void* W2s;
  const float* s1s; const float* s3s; const float* s2s;
  float* y;
  int32_t* topk_idx; float* topk_w; int32_t* counts; int32_t* offsets;
  uint16_t* H;            // [segments, 16, 3, d_ff]
  float* Yp;              // [pieces, T, d]
  int32_t* ctr;           // counters, zeroed by the router launch
  int T, d, E, k, d_ff, capacity, G, M, has_shared, weigh_shared, splits, slots;
  int ahead;              // gate/up tickets are fetched an item ahead
};

// Counters, each in a 128-byte line of its own (atomics and polls of one line are
// served one after the other): gate/up tickets, down tickets, segments, row tiles.
constexpr int kLine = 32;
constexpr int kCtrTicket = 0, kCtrDown = kLine, kCtrSeg = 2 * kLine;
__host__ __device__ inline int few_counters(int segs, int d) {
  return kCtrSeg + (segs + (d + kDownRowsMin - 1) / kDownRowsMin) * kLine;
}

// ---------------------------------------------------------------- router
// partial[t, s, e] = sum over k in split s of x[t, k] W_g[k, e], in fp32.  A
// workgroup takes 16 experts and one split, its waves a quarter of the split
// each.  The fp32 gate is the sum of three bf16 planes (packed beforehand, or
// split here), so each product is exact in fp32.
constexpr int kRouterWaves = 4;
template <bool PACKED>
__global__ __launch_bounds__(kRouterWaves * 64) void few_router_kernel(
    const uint16_t* __restrict__ x, const void* __restrict__ W_g, float* __restrict__ partial,
    int32_t* __restrict__ ctr, int nctr, int T, int d, int E, int E_pad) {
  __shared__ float red[kRouterWaves][256];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = uniform(tid >> 6);
  {  // the counters, spread over the workgroups
    const int b = (blockIdx.y * gridDim.x + blockIdx.x) * kRouterWaves * 64;
    for (int i = b; i < nctr; i += gridDim.x * gridDim.y * kRouterWaves * 64)
      if (i + tid < nctr) ctr[i + tid] = 0;
  }
  const int S = gridDim.y, split = blockIdx.y, e0 = blockIdx.x * 16;
  const int r = lane & 15, g = lane >> 4;
  const int steps = d / 32;
  const int b0 = steps * split / S, b1 = steps * (split + 1) / S;
  const StepMap<WS_BF16> map{0};
  const uint32_t aoff[1] = {r < T ? (uint32_t)r * (uint32_t)d * 2u + map.lane_a(g) : kNowhere};
  const rsrc_t xr = buffer_of(x, (int64_t)T * d * 2);
  f32x4 acc[3][1];
  zero_frags(acc);
  if constexpr (PACKED) {
    const int64_t plane = (int64_t)E_pad * d * 2;
    const char* base = (const char*)W_g + (int64_t)e0 * d * 2;
    const rsrc_t wr[3] = {buffer_of(base, (int64_t)d * 32), buffer_of(base + plane, (int64_t)d * 32),
                          buffer_of(base + 2 * plane, (int64_t)d * 32)};
    stream_rows<WS_BF16, 3, 1, 1, 4, kLoadPlain>(
        map, wr, (uint32_t)r * (uint32_t)d * 2u + map.lane_w(g), xr, aoff, 0u,
        StepShare(b0, b1, wave, kRouterWaves, 0, 0), acc, [] {});
  } else {
    const float* W = (const float*)W_g + min(e0 + r, E - 1);
    for (int s = uniform(b0 + wave); s < b1; s += kRouterWaves) {
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = W[(int64_t)(s * 32 + g * 8 + i) * E];
      bf16x8 pl[3];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t h = f32_to_bf16_bits_any(v[i]);
        const float r1 = v[i] - bf16_bits_to_f32(h);
        const uint32_t m = f32_to_bf16_bits_any(r1);
        const uint32_t l = f32_to_bf16_bits_any(r1 - bf16_bits_to_f32(m));
        pl[0][i] = __builtin_bit_cast(__bf16, (uint16_t)h);
        pl[1][i] = __builtin_bit_cast(__bf16, (uint16_t)m);
        pl[2][i] = __builtin_bit_cast(__bf16, (uint16_t)l);
      }
      const bf16x8 a = __builtin_bit_cast(
          bf16x8, __builtin_amdgcn_raw_buffer_load_b128(xr, aoff[0] + s * 64u, 0, kLoadPlain));
#pragma unroll
      for (int p = 0; p < 3; ++p)
        acc[p][0] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(pl[p], a, acc[p][0], 0, 0, 0);
    }
  }
  *(f32x4*)&red[wave][r * 16 + g * 4] = acc[0][0] + (acc[1][0] + acc[2][0]);
  __syncthreads();
  // entry: token column tid / 16, expert row tid % 16
  const int t = tid >> 4, e = e0 + (tid & 15);
  float v = 0.f;
#pragma unroll
  for (int w = 0; w < kRouterWaves; ++w) v += red[w][tid];
  if (t < T && e < E) partial[((int64_t)t * S + split) * E + e] = v;
}

// ---------------------------------------------------------------- hand-over
// What one workgroup hands to another (h, partial outputs) is stored with
// agent-scope atomic stores and read with agent-scope loads: both go to the point
// where all XCDs meet, so nothing has to be flushed from or dropped in an L2
// (flushing per item cost 110 us of 420 at one token of the Mixtral widths), and
// a count may follow as soon as the stores are acknowledged.  That wait is inline
// assembly so that it stands where it is written.
__device__ __forceinline__ void wait_stores() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

template <typename V>
__device__ __forceinline__ void put(V* p, V v) {
  __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
template <typename V>
__device__ __forceinline__ V get(const V* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Count one arrival after this workgroup's handed-over stores.  Called by all
// threads; the count before it is left in *old (LDS), to be read after a
// barrier.
__device__ __forceinline__ void arrive(int32_t* c, int32_t* old) {
  wait_stores();
  __syncthreads();
  if (threadIdx.x == 0)
    *old = __hip_atomic_fetch_add(c, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Wait until a counter that lower tickets bring to `target` is there; called by
// all threads.  One wave polls, with all lanes (so its loop is a scalar one) and
// with pauses: polls and arrivals queue up at the counter's line.
__device__ __forceinline__ void wait_for(const int32_t* c, int target) {
  if (uniform(threadIdx.x >> 6) == 0)
    while (uniform(get(c)) < target) __builtin_amdgcn_s_sleep(8);
  __syncthreads();
}

// ---------------------------------------------------------------- LDS
struct FewLds {
  float* red;       // [kWaves][4][256] partial tiles of the waves
  uint32_t* mask;   // [E] tokens that chose the expert, << 16 those kept
  int32_t* seg_e;   // [E] touched experts in increasing order
  int32_t* idx;     // [T*k] chosen experts
  float* w;         // [T*k] their weights
  float* shw;       // [16] the shared expert's weight
  int32_t* misc;    // [16]
};

__host__ __device__ inline size_t few_lds_bytes(int T, int E, int k) {
  return 4 * ((size_t)kWaves * 4 * 256 + 2 * (size_t)E + 2 * (size_t)T * k + 32);
}

__device__ __forceinline__ FewLds few_lds(float* b, int T, int E, int k) {
  FewLds L;
  L.red = b;                      b += kWaves * 4 * 256;
  L.mask = (uint32_t*)b;          b += E;
  L.seg_e = (int32_t*)b;          b += E;
  L.idx = (int32_t*)b;            b += T * k;
  L.w = b;                        b += T * k;
  L.shw = b;                      b += 16;
  L.misc = (int32_t*)b;
  return L;
}

// ---------------------------------------------------------------- top-k
// Ordered logit, never 0 (0: not to be chosen).
__device__ __forceinline__ uint32_t order_bits(float v) {
  return max((uint32_t)(topk_key(v, 0) >> 32), 1u);
}
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v = max(v, (uint32_t)__shfl_xor((int)v, o, 64));
  return v;
}

// One wave selects the experts of tokens t0, t0 + step, .. (NT of them, those
// below T): lane l holds experts l, l + 64, ..  Same rule as topk_kernel: the
// largest logit, equal logits the lower index; groups by their largest logit.
template <int EPL, int NT>
__device__ __forceinline__ void route_tokens(const FewParams& p, const FewLds& L, int t0, int step,
                                             int lane) {
  uint32_t key[NT][EPL];
  float v[NT][EPL];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int i = 0; i < EPL; ++i) v[n][i] = 0.f;
#pragma unroll EPL > 4 ? 1 : kMaxSplits
  for (int s = 0; s < kMaxSplits; ++s)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        const float part = p.partial[((int64_t)min(t0 + n * step, p.T - 1) * p.splits +
                                      min(s, p.splits - 1)) * p.E + min(lane + i * 64, p.E - 1)];
        v[n][i] += s < p.splits ? part : 0.f;
      }
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const float b = p.b_g ? p.b_g[min(lane + i * 64, p.E - 1)] : 0.f;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      if (p.b_g) v[n][i] += b;
      key[n][i] = lane + i * 64 < p.E ? order_bits(v[n][i]) : 0u;
    }
  }
  // the best key's lowest expert (uniform)
  auto best_of = [&](const uint32_t (&c)[EPL], uint32_t& top) __attribute__((always_inline)) {
    uint32_t b = 0;
#pragma unroll
    for (int i = 0; i < EPL; ++i) b = max(b, c[i]);
    top = wave_max(b);
    int e = 0;
#pragma unroll
    for (int i = EPL - 1; i >= 0; --i) {
      const uint64_t at = __ballot(c[i] == top);
      if (at) e = i * 64 + __builtin_ctzll(at);
    }
    return min(e, p.E - 1);
  };
  if (p.G > 1) {
    const int gs = p.E / p.G;
    int grp[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) grp[i] = min((lane + i * 64) / gs, 63);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      uint64_t kept = 0;
      for (int m = 0; m < p.M; ++m) {
        uint32_t open[EPL], top;
#pragma unroll
        for (int i = 0; i < EPL; ++i) open[i] = ((kept >> grp[i]) & 1) ? 0u : key[n][i];
        kept |= 1ull << min(best_of(open, top) / gs, 63);
      }
#pragma unroll
      for (int i = 0; i < EPL; ++i)
        if (!((kept >> grp[i]) & 1)) key[n][i] = 0;
    }
  }
  int my_e[NT];
  float my_v[NT], vmax[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    my_e[n] = 0;
    my_v[n] = vmax[n] = 0.f;
  }
  for (int j = 0; j < p.k; ++j)
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      uint32_t top;
      const int e = best_of(key[n], top);
      const float val = key_value((uint64_t)top << 32);
      if (j == 0) vmax[n] = val;
      if (lane == j) { my_e[n] = e; my_v[n] = val; }
#pragma unroll
      for (int i = 0; i < EPL; ++i)
        if (lane + i * 64 == e) key[n][i] = 0;
    }
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int t = t0 + n * step;
    const float ex = lane < p.k ? expf(my_v[n] - vmax[n]) : 0.f;
    const float den = group_sum<64>(ex);
    if (t < p.T && lane < p.k) {
      L.idx[t * p.k + lane] = my_e[n];
      L.w[t * p.k + lane] = ex / den;
    }
  }
}

// Selection and grouping of all tokens, by each workgroup for itself: an
// expert's tokens are a bit mask, the capacity keeps its lowest bits (token
// order), the touched experts are a compaction over E.  Returns their number.
// The first workgroup writes the routing outputs.
__device__ __forceinline__ int route_and_group(const FewParams& p, const FewLds& L) {
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = uniform(tid >> 6);
  const int A = p.T * p.k;
  for (int b = 0; b < p.E; b += kThreads)
    if (b + tid < p.E) L.mask[b + tid] = 0;
  if (wave < p.T) {
    if (p.E > 256) {
      for (int t = wave; t < p.T; t += kWaves) route_tokens<16, 1>(p, L, t, kWaves, lane);
    } else if (p.E > 64) {
      route_tokens<4, kCols / kWaves>(p, L, wave, kWaves, lane);
    } else {
      route_tokens<1, kCols / kWaves>(p, L, wave, kWaves, lane);
    }
  }
  __syncthreads();
  for (int b = 0; b < A; b += kThreads)
    if (b + tid < A) atomicOr(&L.mask[L.idx[b + tid]], 1u << ((b + tid) / p.k));
  __syncthreads();
  const int per = (p.E + kThreads - 1) / kThreads;
  int mine = 0;  // kept rows << 16 | touched experts
  for (int i = 0; i < per; ++i) {
    const int e = tid * per + i;
    if (e < p.E) {
      const uint32_t chosen = L.mask[e];
      uint32_t kept = chosen;
      if (p.capacity >= 0) {
        uint32_t rest = chosen;
        kept = 0;
#pragma unroll
        for (int c = 0; c < kCols; ++c) {
          const uint32_t low = rest & (0u - rest);
          if (c < p.capacity) kept |= low;
          rest ^= low;
        }
      }
      L.mask[e] = chosen | kept << 16;
      mine += (__popc(kept) << 16) + (kept != 0);
    }
  }
  int incl = mine;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int v = __shfl_up(incl, o, 64);
    if (lane >= o) incl += v;
  }
  if (lane == 63) L.misc[8 + wave] = incl;
  __syncthreads();
  int run = incl - mine, total = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    if (w < wave) run += L.misc[8 + w];
    total += L.misc[8 + w];
  }
  const bool report = blockIdx.x == 0;
  for (int i = 0; i < per; ++i) {
    const int e = tid * per + i;
    if (e < p.E) {
      const uint32_t m = L.mask[e];
      if (m >> 16) L.seg_e[run & 0xFFFF] = e;
      if (report) {
        p.counts[e] = __popc(m & 0xFFFFu);
        p.offsets[e] = run >> 16;
        if (e == p.E - 1) p.offsets[p.E] = total >> 16;
      }
      run += (__popc(m >> 16) << 16) + ((m >> 16) != 0);
    }
  }
  if (report)
    for (int b = 0; b < A; b += kThreads)
      if (b + tid < A) {
        p.topk_idx[b + tid] = L.idx[b + tid];
        p.topk_w[b + tid] = L.w[b + tid];
      }
  if (p.has_shared && tid < p.T) {
    float w = 1.f;
    if (p.weigh_shared)
      for (int j = 0; j < p.k; ++j)
        if (!((L.mask[L.idx[tid * p.k + j]] >> (16 + tid)) & 1)) w += L.w[tid * p.k + j];
    L.shw[tid] = w;
  }
  __syncthreads();
  return total & 0xFFFF;
}

// One segment: a touched expert or (e = -1) the shared one, and its tokens.
struct Segment {
  int e;
  uint32_t tokens;
};

__device__ __forceinline__ Segment segment(const FewParams& p, const FewLds& L, int seg) {
  if (p.has_shared && seg == 0) return {-1, (1u << p.T) - 1};
  Segment s;
  s.e = uniform(L.seg_e[seg - p.has_shared]);
  s.tokens = (uint32_t)uniform((int)(L.mask[s.e] >> 16));
  return s;
}

// ---------------------------------------------------------------- gate / up
__device__ __forceinline__ int next_ticket(int32_t* c) {
  return __hip_atomic_fetch_add(c, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// The queue as a workgroup sees it; all values are the same in every thread.
// Gate/up: the ticket it works on and the next one, which it holds already where
// there are several items per workgroup (`ahead`: neither the fetch nor the next
// item's first weight loads wait for the present item's end; with fewer items a
// workgroup would hold two while another has none: 64 narrow experts, one
// token: 50 us against 68).  A ticket past the gate/up
// items means that all of these are taken: the workgroup goes on to the down
// items, which have a counter of their own and are fetched when needed (few and
// long, a workgroup must not hold two while another has none).
struct Queue {
  int q, qn;
  int nseg, tiles, pieces, ready;
};

// Gate/up items, as long as the workgroup's tickets are such: 16 U hidden columns
// f0 .. of one segment, U row tiles of W1 and the same of W3; silu, product and
// routing weight in the reduction.  Each wave streams its part of the rows in
// blocks of PD steps; a step's registers are refilled, as soon as its MFMAs have
// read them, with the same step of the next block, which may be the next item's
// first: the weight stream does not pause between items.  Steps past the end
// load zeros from nowhere.
template <int WQ, int U>
__device__ __forceinline__ void gate_up_items(const FewParams& p, const FewLds& L, Queue& Q) {
  constexpr int LS = StreamFmt<WQ>::LS, MF = StreamFmt<WQ>::MF;
  constexpr int PD = WQ == WS_BF16 ? 8 : 4;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = uniform(tid >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int64_t rowb = weight_bytes<WQ>(p.d);
  const rsrc_t xr = buffer_of(p.x, (int64_t)p.T * p.d * 2);
  const int steps = p.d / LS;
  const StepMap<WQ> map{steps % 2 == 0 ? 1 : 0};
  const uint32_t wlane = (uint32_t)(r * rowb) + map.lane_w(g), tile = (uint32_t)(16 * rowb);
  const StepShare share(0, steps, wave, kWaves, map.pair, 0);
  const int blocks = (share.count + PD - 1) / PD;
  const int up_items = Q.nseg * Q.tiles;
  u32x4 w[PD][2 * U], a[PD][MF];

  struct Item {
    int seg, e, f0;
    uint32_t tokens, aoff;
    rsrc_t w1, w3;
  };
  auto item = [&](int q) __attribute__((always_inline)) {
    Item it;
    it.seg = q / Q.tiles;
    it.f0 = (q - it.seg * Q.tiles) * (16 * U);
    const Segment sg = segment(p, L, it.seg);
    it.e = sg.e;
    it.tokens = sg.tokens;
    const int64_t moff = ((sg.e < 0 ? 0 : (int64_t)sg.e * p.d_ff) + it.f0) * rowb;
    it.w1 = buffer_of((const char*)(sg.e < 0 ? p.W1s : p.W1) + moff, 16 * U * rowb);
    it.w3 = buffer_of((const char*)(sg.e < 0 ? p.W3s : p.W3) + moff, 16 * U * rowb);
    it.aoff = (sg.tokens >> r) & 1 ? (uint32_t)r * (uint32_t)p.d * 2u + map.lane_a(g) : kNowhere;
    return it;
  };
  // the wave's step j of an item into register slot i (past the end, or j < 0: zeros)
  auto load = [&](int i, const Item& it, int j) __attribute__((always_inline)) {
    const int s = share.step(max(j, 0));
    const bool in = j >= 0 && j < share.count && s < share.end;
    const uint32_t o = in ? wlane + map.w(s) : kNowhere;
#pragma unroll
    for (int t = 0; t < U; ++t) {
      w[i][2 * t] = __builtin_amdgcn_raw_buffer_load_b128(it.w1, o + t * tile, 0, kLoadPlain);
      w[i][2 * t + 1] = __builtin_amdgcn_raw_buffer_load_b128(it.w3, o + t * tile, 0, kLoadPlain);
    }
    const uint32_t ao = in ? it.aoff + map.a(s) : kNowhere;
#pragma unroll
    for (int m = 0; m < MF; ++m)
      a[i][m] = __builtin_amdgcn_raw_buffer_load_b128(xr, ao + m * 16, 0, kLoadPlain);
  };

  Item cur = item(Q.q);
#pragma unroll
  for (int i = 0; i < PD; ++i) load(i, cur, i);
  for (;;) {
    int ticket = 0;
    if (tid == 0 && p.ahead) ticket = next_ticket(p.ctr + kCtrTicket);
    const bool more = p.ahead && Q.qn < up_items;
    const Item nxt = item(more ? Q.qn : Q.q);
    f32x4 acc[2 * U];
#pragma unroll
    for (int t = 0; t < 2 * U; ++t) acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
    auto compute = [&](int i) __attribute__((always_inline)) {
#pragma unroll
      for (int m = 0; m < MF; ++m) {
        const bf16x8 b = __builtin_bit_cast(bf16x8, a[i][m]);
#pragma unroll
        for (int t = 0; t < 2 * U; ++t)
          acc[t] =
              __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen<WQ>(w[i][t], m), b, acc[t], 0, 0, 0);
      }
    };
    for (int blk = 1; blk < blocks; ++blk)
#pragma unroll
      for (int i = 0; i < PD; ++i) {
        compute(i);
        load(i, cur, blk * PD + i);
      }
#pragma unroll
    for (int i = 0; i < PD; ++i) {
      compute(i);
      load(i, nxt, more ? i : -1);
    }
#pragma unroll
    for (int t = 0; t < 2 * U; ++t)
      *(f32x4*)&L.red[(wave * 2 * U + t) * 256 + r * 16 + g * 4] = acc[t];
    // entry: row tile tid / 256, token column, hidden column (first 256 U threads)
    const int half = tid >> 8, c = (tid >> 4) & 15;
    float wgt = 1.f;
    if (cur.e >= 0) {
      for (int j = 0; j < p.k; ++j)
        if (c < p.T && L.idx[c * p.k + j] == cur.e) wgt = L.w[c * p.k + j];
    } else if (p.weigh_shared && c < p.T) {
      wgt = L.shw[c];
    }
    float sc1 = 1.f, sc3 = 1.f;
    if (WQ != WS_BF16) {
      const int gi = cur.f0 / kFp8Group;
      sc1 = kWeightUnit<WQ> *
            (cur.e < 0 ? p.s1s[gi] : p.s1[(int64_t)cur.e * (p.d_ff / kFp8Group) + gi]);
      sc3 = kWeightUnit<WQ> *
            (cur.e < 0 ? p.s3s[gi] : p.s3[(int64_t)cur.e * (p.d_ff / kFp8Group) + gi]);
    }
    __syncthreads();
    if (wave < 4 * U) {
      float ga = 0.f, up = 0.f;
#pragma unroll
      for (int v = 0; v < kWaves; ++v) {
        ga += L.red[((v * U + half) * 2) * 256 + (tid & 255)];
        up += L.red[((v * U + half) * 2 + 1) * 256 + (tid & 255)];
      }
      ga *= sc1;
      up *= sc3;
      const float h = ga / (1.f + __expf(-ga)) * up * wgt;
      uint32_t hb, mb, lb;
      split3(h, hb, mb, lb);
      // two neighbouring columns per store, by the even lane
      const uint32_t hv = hb | (uint32_t)__shfl_xor((int)hb, 1, 64) << 16;
      const uint32_t mv = mb | (uint32_t)__shfl_xor((int)mb, 1, 64) << 16;
      const uint32_t lv = lb | (uint32_t)__shfl_xor((int)lb, 1, 64) << 16;
      if (((cur.tokens >> c) & 1) && !(tid & 1)) {
        uint32_t* o =
            (uint32_t*)(p.H + ((int64_t)cur.seg * kCols + c) * 3 * p.d_ff + cur.f0 + half * 16 +
                        (tid & 15));
        put(o, hv);
        put(o + p.d_ff / 2, mv);
        put(o + p.d_ff, lv);
      }
    }
    if (tid == 0) L.misc[0] = ticket;
    arrive(p.ctr + kCtrSeg + cur.seg * kLine, L.misc + 1);
    if (p.ahead) {
      Q.q = Q.qn;
      Q.qn = uniform(L.misc[0]);
      if (!more) return;
      cur = nxt;
    } else {
      if (tid == 0) L.misc[3] = next_ticket(p.ctr + kCtrTicket);
      __syncthreads();
      Q.q = uniform(L.misc[3]);
      if (Q.q >= up_items) return;
      cur = item(Q.q);
#pragma unroll
      for (int i = 0; i < PD; ++i) load(i, cur, i);
    }
  }
}

// ---------------------------------------------------------------- down
// One down item: the output rows of one row tile for one piece of the concatenated
// hidden columns of all segments, the waves sharing each segment's steps; the last
// piece of a row tile to finish adds the pieces up, in piece order.
template <int WQ>
__device__ __forceinline__ void down_item(const FewParams& p, const FewLds& L, Queue& Q, int q) {
  constexpr int kRows = down_rows(WQ), RT = kRows / 16, LS = StreamFmt<WQ>::LS;
  constexpr int PD = WQ == WS_BF16 ? 3 : WQ == WS_FP8 ? 2 : 1;  // steps in flight
  constexpr int HT = 4;  // row tiles reduced at a time (the LDS holds those)
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = uniform(tid >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int pieces = Q.pieces;
  const int ntiles = (p.d + kRows - 1) / kRows, kunits = p.d_ff / 128;
  const int piece = q / ntiles, nt = q - piece * ntiles, n0 = nt * kRows;
  const int64_t rowb = weight_bytes<WQ>(p.d_ff);
  const StepMap<WQ> map{p.d_ff / LS % 2 == 0 ? 1 : 0};
  const int units = Q.nseg * kunits;
  const int lo = uniform(units * piece / pieces), hi = uniform(units * (piece + 1) / pieces);
  // The waves share a segment's steps line by line, unless they are few: then each
  // wave takes a part of the piece of its own (a step or two of each wave per segment
  // pause the stream with every segment: 32 experts of 256 hidden columns, int8, 11
  // tokens, 41 us against 34; 64 of 1408, int4, 16 tokens, 98 against 94; but of 64
  // steps, 32 experts of 2048, bf16, 16 tokens, 616 against 657).
  const int teams = uniform(p.d_ff / LS >= 32 ? 1 : kWaves), size = kWaves / teams;
  const int team = uniform(wave / size);
  if (teams > 1)
    for (int seg = uniform(max(Q.ready, lo / kunits)); seg * kunits < hi; ++seg) {
      wait_for(p.ctr + kCtrSeg + seg * kLine, Q.tiles);
      Q.ready = seg + 1;
    }
  const int u0 = uniform(lo + (hi - lo) * team / teams);
  const int u1 = uniform(lo + (hi - lo) * (team + 1) / teams);
  f32x4 sum[RT][1];
  zero_frags(sum);
  for (int u = u0; u < u1;) {
    const int seg = u / kunits, k0 = u - seg * kunits;
    const int k1 = min(kunits, k0 + u1 - u);
    const Segment sg = segment(p, L, seg);
    const char* b = (const char*)(sg.e < 0 ? p.W2s : p.W2) +
                    ((sg.e < 0 ? 0 : (int64_t)sg.e * p.d) + n0) * rowb;
    rsrc_t wr[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i)  // (d is a multiple of 64: whole row tiles)
      wr[i] = buffer_of(b + i * 16 * rowb, n0 + i * 16 < p.d ? 16 * rowb : 0);
    const uint32_t aoff[1] = {
        (sg.tokens >> r) & 1 ? (uint32_t)r * 6u * (uint32_t)p.d_ff + map.lane_a(g) : kNowhere};
    const StepShare share(k0 * (128 / LS), k1 * (128 / LS), wave % size, size, map.pair, nt);
    const rsrc_t hr =
        buffer_of(p.H + (int64_t)seg * kCols * 3 * p.d_ff, (int64_t)kCols * 6 * p.d_ff);
    auto ready = [&]() __attribute__((always_inline)) {
      if (teams == 1 && seg >= Q.ready) {  // segments below `ready` were waited for before
        wait_for(p.ctr + kCtrSeg + seg * kLine, Q.tiles);
        Q.ready = seg + 1;
      }
    };
    const uint32_t wlane = (uint32_t)(r * rowb) + map.lane_w(g), plane = (uint32_t)p.d_ff * 2u;
    // A column without the segment keeps its sum: its products are zeros times the
    // weights, which need not be finite.
    const bool own = (sg.tokens >> r) & 1;
    if constexpr (WQ == WS_BF16) {
      f32x4 kept[RT];
#pragma unroll
      for (int i = 0; i < RT; ++i) kept[i] = sum[i][0];
      stream_rows<WQ, RT, 1, 3, PD, kLoadAgent>(map, wr, wlane, hr, aoff, plane, share, sum, ready);
#pragma unroll
      for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) sum[i][0][c] = own ? sum[i][0][c] : kept[i][c];
    } else {
      f32x4 acc[RT][1];
      zero_frags(acc);
      stream_rows<WQ, RT, 1, 3, PD, kLoadAgent>(map, wr, wlane, hr, aoff, plane, share, acc, ready);
      const float sc = kWeightUnit<WQ> *
                       (sg.e < 0 ? p.s2s[nt] : p.s2[(int64_t)sg.e * (p.d / kFp8Group) + nt]);
#pragma unroll
      for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c)
          sum[i][0][c] = own ? fmaf(sc, acc[i][0][c], sum[i][0][c]) : sum[i][0][c];
    }
    u += k1 - k0;
  }
  static_assert(WQ == WS_BF16 || kRows == kFp8Group, "one scale per down item");
  // entries: token column c, output rows n0 + 16 * (h * HT + i0 + i) + tid % 16
  const int c = (tid >> 4) & 15, i0 = (tid >> 8) * (HT / 2);
  const int64_t o = (int64_t)c * p.d + n0 + i0 * 16 + (tid & 15);
  const int64_t stride = (int64_t)p.T * p.d;
  float* out = pieces == 1 ? p.y : p.Yp + piece * stride;
#pragma unroll
  for (int h = 0; h < RT / HT; ++h) {
    if (h) __syncthreads();
#pragma unroll
    for (int i = 0; i < HT; ++i)
      *(f32x4*)&L.red[(wave * HT + i) * 256 + r * 16 + g * 4] = sum[h * HT + i][0];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < HT / 2; ++i) {
      float v = 0.f;
#pragma unroll
      for (int u = 0; u < kWaves; ++u) v += L.red[(u * HT + i0 + i) * 256 + (tid & 255)];
      if (c < p.T && n0 + (h * HT + i0 + i) * 16 < p.d) put(out + o + (h * HT + i) * 16, v);
    }
  }
  if (pieces == 1) return;
  arrive(p.ctr + kCtrSeg + (Q.nseg + nt) * kLine, L.misc + 1);
  __syncthreads();
  if (uniform(L.misc[1]) == pieces - 1 && c < p.T) {
#pragma unroll
    for (int h = 0; h < RT / HT; ++h)
#pragma unroll
      for (int i = 0; i < HT / 2; ++i) {
        if (n0 + (h * HT + i0 + i) * 16 >= p.d) continue;
        float part[kMaxPieces], v = 0.f;
#pragma unroll
        for (int j = 0; j < kMaxPieces; ++j)
          part[j] = j < pieces ? get(p.Yp + j * stride + o + (h * HT + i) * 16) : 0.f;
#pragma unroll
        for (int j = 0; j < kMaxPieces; ++j) v += part[j];
        p.y[o + (h * HT + i) * 16] = v;
      }
  }
}

// ---------------------------------------------------------------- the layer
template <int WQ, int U>
__global__ __launch_bounds__(kThreads, 2) void few_layer_kernel(FewParams p) {
  extern __shared__ __align__(16) float lds[];
  const FewLds L = few_lds(lds, p.T, p.E, p.k);
  const int tid = threadIdx.x;
  const int ntiles = (p.d + down_rows(WQ) - 1) / down_rows(WQ);
  // by the last wave: it has the fewest tokens to select, and loads return behind
  // these contended atomics
  constexpr int kFetch = kThreads - 64;
  int first = 0, second = 0;
  if (tid == kFetch) {
    first = next_ticket(p.ctr + kCtrTicket);
    if (p.ahead) second = next_ticket(p.ctr + kCtrTicket);
  }
  Queue Q;
  Q.nseg = uniform(route_and_group(p, L)) + p.has_shared;
  Q.tiles = p.d_ff / (16 * U);
  // pieces per row tile: one round of down items over the workgroups
  Q.pieces = uniform(max(1, min(min(kMaxPieces, Q.nseg * (p.d_ff / 128)), p.slots / ntiles)));
  Q.ready = 0;
  if (tid == kFetch) {
    L.misc[0] = first;
    L.misc[1] = second;
  }
  __syncthreads();
  Q.q = uniform(L.misc[0]);
  Q.qn = uniform(L.misc[1]);
  __syncthreads();
  if (Q.q < Q.nseg * Q.tiles) gate_up_items<WQ, U>(p, L, Q);
  for (;;) {
    __syncthreads();  // the item's LDS and the ticket's reads are done
    if (tid == 0) L.misc[2] = next_ticket(p.ctr + kCtrDown);
    __syncthreads();
    const int q = uniform(L.misc[2]);
    if (q >= ntiles * Q.pieces) break;
    Q.ready = uniform(Q.ready);
    down_item<WQ>(p, L, Q, q);
  }
}

template <int WQ>
void launch_layer(const FewParams& p, int U, int blocks, size_t lds, hipStream_t st) {
  if constexpr (WQ != WS_BF16) {
    if (U == 2) {
      few_layer_kernel<WQ, 2><<<blocks, kThreads, lds, st>>>(p);
      return;
    }
  }
  few_layer_kernel<WQ, 1><<<blocks, kThreads, lds, st>>>(p);
}

// T == 0: zero counts and offsets.
__global__ void few_empty_kernel(int32_t* counts, int32_t* offsets, int E) {
  for (int e = threadIdx.x; e <= E; e += blockDim.x) {
    if (e < E) counts[e] = 0;
    offsets[e] = 0;
  }
}

// K splits of the router: enough workgroups to read the gate at once, but no
// more partial logits than every workgroup of the second launch can sum.
int few_splits(const moe_shape& s) { return std::max(1, std::min(kMaxSplits, s.d / 128)); }

// Most segments a call can touch.
int64_t few_segments(const moe_shape& s) {
  return std::min<int64_t>(s.E, s.T * s.top_k) + (s.has_shared ? 1 : 0);
}

size_t align256(size_t v) { return (v + 255) & ~(size_t)255; }

struct FewLayout {
  size_t off_ctr, off_partial, off_H, off_Yp, total;
};

FewLayout few_layout(const moe_shape& s) {
  FewLayout L{};
  const int64_t segs = few_segments(s);
  size_t off = 0;
  L.off_ctr = off;
  off = align256(off + (size_t)few_counters((int)segs, s.d) * 4);
  L.off_partial = off;
  off = align256(off + (size_t)s.T * few_splits(s) * s.E * 4);
  L.off_H = off;
  off = align256(off + (size_t)segs * kCols * 3 * s.d_ff * 2);
  L.off_Yp = off;
  off = align256(off + (size_t)kMaxPieces * s.T * s.d * 4);
  L.total = off;
  return L;
}

}  // namespace

size_t few_workspace_bytes(const moe_shape& s) { return few_layout(s).total; }

hipError_t launch_forward_few(const moe_shape& s, const void* x, const float* W_g, const float* b_g,
                              const moe_weights& w, float* y, int32_t* topk_idx, float* topk_w,
                              int32_t* counts, int32_t* offsets, void* ws, hipStream_t st) {
  if (s.T == 0) {
    few_empty_kernel<<<1, 256, 0, st>>>(counts, offsets, s.E);
    return hipGetLastError();
  }
  const FewLayout L = few_layout(s);
  char* b = (char*)ws;
  int32_t* ctr = (int32_t*)(b + L.off_ctr);
  float* partial = (float*)(b + L.off_partial);
  const dim3 grid((unsigned)((s.E + 15) / 16), (unsigned)few_splits(s));
  const int64_t segs = few_segments(s);
  const int nctr = few_counters((int)segs, s.d);
  if (s.router_packed)
    few_router_kernel<true><<<grid, kRouterWaves * 64, 0, st>>>(
        (const uint16_t*)x, W_g, partial, ctr, nctr, (int)s.T, s.d, s.E, router_mfma_epad(s));
  else
    few_router_kernel<false><<<grid, kRouterWaves * 64, 0, st>>>(
        (const uint16_t*)x, W_g, partial, ctr, nctr, (int)s.T, s.d, s.E, 0);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  FewParams p{};
  p.x = (const uint16_t*)x;
  p.partial = partial;
  p.b_g = b_g;
  p.W1 = w.W1; p.W3 = w.W3; p.W2 = w.W2; p.s1 = w.s1; p.s3 = w.s3; p.s2 = w.s2;
  p.W1s = w.W1s; p.W3s = w.W3s; p.W2s = w.W2s; p.s1s = w.s1s; p.s3s = w.s3s; p.s2s = w.s2s;
  p.y = y; p.topk_idx = topk_idx; p.topk_w = topk_w; p.counts = counts; p.offsets = offsets;
  p.H = (uint16_t*)(b + L.off_H);
  p.Yp = (float*)(b + L.off_Yp);
  p.ctr = ctr;
  p.T = (int)s.T; p.d = s.d; p.E = s.E; p.k = s.top_k; p.d_ff = s.d_ff; p.capacity = s.capacity;
  p.G = s.n_groups; p.M = s.topk_groups; p.has_shared = s.has_shared ? 1 : 0;
  p.weigh_shared = s.overflow == MOE_OVERFLOW_SHARED && s.capacity >= 0 ? 1 : 0;
  p.splits = (int)grid.y;
  p.slots = current_device_cus();
  const int64_t up16 = segs * (s.d_ff / 16);
  // Items of 32 hidden columns where quantised weights give a workgroup several:
  // fewer reductions, and x read from L2 half as often (16 tokens, Mixtral widths,
  // int4: 259 us against 239, int8: 358 against 343); with fewer items the split is
  // too coarse (one token, 32 experts of 2048, int4: 92 us against 102), and bf16
  // weights take long enough to hide both (16 tokens: 574 against 577).
  const int U = s.w_dtype != MOE_DT_BF16 && up16 >= 8 * (int64_t)p.slots ? 2 : 1;
  // no more workgroups than the queue can have items
  const int64_t items = std::max<int64_t>(up16 / U, (s.d + kDownRowsMin - 1) / kDownRowsMin * kMaxPieces);
  const int blocks = (int)std::min<int64_t>(p.slots, items);
  p.ahead = up16 / U > 3 * blocks ? 1 : 0;
  const size_t lds = few_lds_bytes(p.T, p.E, p.k);
  switch (s.w_dtype) {
    case MOE_DT_BF16: launch_layer<WS_BF16>(p, U, blocks, lds, st); break;
    case MOE_DT_FP8_E4M3: launch_layer<WS_FP8>(p, U, blocks, lds, st); break;
    case MOE_DT_INT8: launch_layer<WS_INT8>(p, U, blocks, lds, st); break;
    case MOE_DT_INT4: launch_layer<WS_INT4>(p, U, blocks, lds, st); break;
    default: return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

}  // namespace moe
