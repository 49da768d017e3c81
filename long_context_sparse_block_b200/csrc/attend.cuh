// What the attention kernels share: the launch's parameters, the units of work of
// a packed batch, the workspace of units that were cut into parts and the kernel
// that joins them.
#pragma once

#include <algorithm>

#include "internal.h"

namespace misa {
namespace {

constexpr int kTile = 128;       // keys per tile of the dense form
constexpr int kPartRows = 256;   // workspace rows of a part (two slots of 128)
constexpr float kRaise = 8.0f;   // log2 of the largest weight before m is raised
constexpr int kMaxCtas = 256;
constexpr int kRowHeads = 16;    // list form: query heads of a key head that the row kernel takes

struct AttParams {
  const uint16_t* Q;        // [n_tok, H, D]
  const uint16_t* kp;       // [n_pages, page, Hkv, D]
  const uint16_t* vp;
  const int32_t* bts;       // [n_seq, max_blocks]
  const int32_t* cu_q;      // [n_seq + 1]
  const int32_t* lens;      // [n_seq]
  const int32_t* seq_of;    // list form: [n_tok]
  const int32_t* positions; // list form: [n_tok]
  const int32_t* idx;       // list form: [n_tok, k]
  uint16_t* out;            // [n_tok, H, D]
  float* lse;               // [n_tok, H], nullable
  int64_t n_pages;
  int64_t key_rows;
  int max_blocks;
  int page_shift;
  int n_seq;
  int n_tok;
  int H;
  int Hkv;
  int G;
  int T;                    // tokens of a slot: 128 / G
  int g_inv;                // 65536 / G + 1: x / G == x * g_inv >> 16 for x < 384, G <= 128
  int window;               // 0: none
  int sinks;
  int k;
  float c;                  // scale * log2(e)
  int workers;              // CTAs (row kernel: warps) that share the line
  uint64_t w_inv;           // 2^64 / workers + 1
  // workspace
  int4* head;               // [ctas][2]: what each CTA left in parts
  float* ml;                // [2 ctas][256][2]
  float* po;                // [2 ctas][256][D]
  DevCtl ctl;
};

// ---- units -------------------------------------------------------------------

struct Unit {
  int b;       // sequence (list form: unused)
  int m;       // row block (list form: token)
  int j;       // key head
  int64_t off; // cost already spent of this unit
};

struct SeqInfo {
  int64_t t0;  // first row of the packed batch
  int n;       // new tokens
  int len;     // keys
  int p0;      // position of the first new token
};

__device__ __forceinline__ SeqInfo seq_info(const AttParams& p, int b) {
  SeqInfo s;
  int t0 = __ldg(p.cu_q + b), t1 = __ldg(p.cu_q + b + 1);
  t0 = min(max(t0, 0), p.n_tok);
  t1 = min(max(t1, t0), p.n_tok);
  int64_t len = __ldg(p.lens + b);
  const int64_t cap = static_cast<int64_t>(p.max_blocks) << p.page_shift;
  len = len < 0 ? 0 : len > cap ? cap : len;
  s.t0 = t0;
  s.n = t1 - t0;
  s.len = static_cast<int>(len);
  s.p0 = s.len - s.n;
  return s;
}

// A unit's rows are the G heads of 2 T tokens: two slots of T tokens, head by head.
__device__ __forceinline__ int64_t row_blocks(const AttParams& p, const SeqInfo& s) {
  return (static_cast<int64_t>(s.n) + 2 * p.T - 1) / (2 * p.T);
}

// Cost of block m of a sequence and its sum over blocks 0..m-1: about the keys it
// passes over, and what a unit costs beside them (loading and storing its rows:
// measured at three to four tiles).  Only the balance depends on it.
constexpr int kUnitCost = 4 * kTile;
__device__ __forceinline__ int64_t cost_base(const SeqInfo& s) { return max(s.p0, 0) + kUnitCost; }
__device__ __forceinline__ int64_t cost_flat(const AttParams& p) {
  return p.window ? static_cast<int64_t>(p.window) + p.sinks + 2 * p.T + kUnitCost
                  : 0x3fffffffffffffffLL;
}
__device__ __forceinline__ int64_t cost_of(const AttParams& p, const SeqInfo& s, int64_t m) {
  return min(cost_base(s) + 2 * p.T * (m + 1), cost_flat(p));
}
__device__ __forceinline__ int64_t cost_before(const AttParams& p, const SeqInfo& s, int64_t m) {
  const int64_t base = cost_base(s), flat = cost_flat(p);
  // blocks below `lin` grow with m, those from it on cost `flat`
  int64_t lin = m;
  if (p.window) lin = min(m, flat > base ? (flat - base) / (2 * p.T) : 0);
  return lin * base + p.T * (lin * (lin + 1)) + (m > lin ? (m - lin) * flat : 0);
}

// Tiles of a unit: `sink` tiles from the start, then tiles lo.. .
struct Tiles {
  int n;     // tiles in all
  int sink;
  int lo;
  int toks;  // tokens of the unit
};

__device__ __forceinline__ Tiles unit_tiles(const AttParams& p, const SeqInfo& s, int m) {
  Tiles t;
  t.toks = min(2 * p.T, s.n - m * 2 * p.T);
  const int p_first = s.p0 + m * 2 * p.T, p_last = p_first + t.toks - 1;
  const int end = p_last < 0 ? 1 : p_last / kTile + 1;  // a unit that sees nothing passes one tile
  t.lo = 0;
  t.sink = 0;
  if (p.window) {
    const int64_t f = static_cast<int64_t>(p_first) - p.window + 1;
    t.lo = f > 0 ? static_cast<int>(f / kTile) : 0;
    t.sink = min((p.sinks + kTile - 1) / kTile, t.lo);
  }
  t.n = t.sink + end - t.lo;
  return t;
}
// The tile at which a cost offset falls.  Every CTA and the joining kernel must
// agree on it, so each operation is rounded on its own; monotone in off.
__device__ __forceinline__ int tile_of(int64_t off, int64_t cost, int n) {
  if (off <= 0) return 0;
  if (off >= cost) return n;
  const float f = __fdiv_rn(__ll2float_rn(off), __ll2float_rn(cost));
  return min(n, __float2int_rd(__fmul_rn(f, __int2float_rn(n))));
}
// Point c of a line of `total` (< 2^48) cut evenly in n <= p.workers; for n =
// p.workers a multiplication by w_inv = 2^64 / workers + 1 stands for the division.
__device__ __forceinline__ int64_t cut(const AttParams& p, int n, int64_t total, int c) {
  if (n == 1) return c > 0 ? total : 0;
  const int64_t q =
      n == p.workers ? static_cast<int64_t>(__umul64hi(static_cast<uint64_t>(total), p.w_inv)) : total / n;
  return q * c + static_cast<int>(total - q * n) * c / n;
}

// ---- small device helpers --------------------------------------------------------

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// log(sum) of a row with reference m (in log2) and sum l.
__device__ __forceinline__ float row_lse(float m, float l) {
  return l > 0.0f ? (m + __log2f(l)) * 0.69314718055994530942f : l == 0.0f ? -INFINITY : l;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(r)
      : "l"(*reinterpret_cast<const uint64_t*>(&a)), "l"(*reinterpret_cast<const uint64_t*>(&b)));
  return *reinterpret_cast<const float2*>(&r);
}
// A unit that worker w (a CTA, or a warp of the row kernel) opens and does not
// finish is summed in parts: w leaves its part in workspace slot 2 w + 1, the
// workers after it that have a tile of the unit theirs in slot 2 e.  They write
//   head[2 w]     x: 1 if w has a part of a unit that an earlier worker opened
//   head[2 w + 1] x: 1 if w opens such a unit, y: its first token in the packed
//                 batch, z: tokens, key head << 16, w: the worker that ends it
// The last worker with a point of the line before `end`:
__device__ __forceinline__ int last_worker(const AttParams& p, int n, int64_t total, int64_t end) {
  int e = static_cast<int>(static_cast<float>(end - 1) / static_cast<float>(total) * n);
  e = min(max(e, 0), n - 1);
  while (e > 0 && cut(p, n, total, e) >= end) --e;
  while (e + 1 < n && cut(p, n, total, e + 1) < end) ++e;
  return e;
}

// Joins the parts of the unit that worker blockIdx.x opened:
//   o = sum_i 2^(m_i - m) o_i / sum_i 2^(m_i - m) l_i,  parts in worker order.
// A warp takes a row.  Latency is what it costs (a few dependent loads), so up to
// four parts, the usual case, are loaded at once; more go by 32, a lane holding a
// part's m and l.
constexpr int kJoinThreads = 256;
constexpr int kJoinWarps = kJoinThreads / 32;
constexpr int kJoinBlocks = 16;  // blocks that share a dense unit's rows

template <int V>
__device__ __forceinline__ void load_part(const float* src, float (&y)[V]) {
  if constexpr (V == 4) {
    const float4 z = *reinterpret_cast<const float4*>(src);
    y[0] = z.x, y[1] = z.y, y[2] = z.z, y[3] = z.w;
  } else {
    const float2 z = *reinterpret_cast<const float2*>(src);
    y[0] = z.x, y[1] = z.y;
  }
}

template <int D>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const AttParams p, int part_rows) {
  const int c = blockIdx.x, lane = lane_id();
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the attention kernel is done
  const int4 open = p.head[2 * c + 1];
  if (!open.x) return;
  const int rows = (open.z & 0xffff) * p.G, j = open.z >> 16, n = open.w - c + 1;
  int x = blockIdx.y * kJoinWarps + warp_id();
  if (x >= rows) return;
  bool has[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) has[i] = i == 0 || (i < n && p.head[2 * (c + i)].x);
  constexpr int V = D / 32;  // elements of a lane
  for (; x < rows; x += gridDim.y * kJoinWarps) {
    const int tok = x * p.g_inv >> 16, hd = x - tok * p.G;
    const int r = tok < p.T ? x : x - p.T * p.G + kTile;  // workspace row: slot 1 starts at 128
    auto at = [&](int i) {  // row of part i
      return static_cast<int64_t>(i == 0 ? 2 * c + 1 : 2 * (c + i)) * part_rows + r;
    };
    float m, l = 0.0f, o[V];
#pragma unroll
    for (int e = 0; e < V; ++e) o[e] = 0.0f;
    if (n <= 4) {
      float pm[4], pl[4], y[4][V];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        pm[i] = -INFINITY;
        pl[i] = 0.0f;
        if (has[i]) {
          const float2 z = *reinterpret_cast<const float2*>(p.ml + 2 * at(i));
          pm[i] = z.x;
          pl[i] = z.y;
          load_part<V>(p.po + at(i) * D + lane * V, y[i]);
        }
      }
      m = fmaxf(fmaxf(pm[0], pm[1]), fmaxf(pm[2], pm[3]));
      const float ref = m == -INFINITY ? 0.0f : m;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (!has[i]) continue;
        const float f = ex2(pm[i] - ref);
        l = fmaf(f, pl[i], l);
#pragma unroll
        for (int e = 0; e < V; ++e) o[e] = fmaf(f, y[i][e], o[e]);
      }
    } else {
      m = -INFINITY;
      for (int i0 = 0; i0 < n; i0 += 32) {
        const int i = i0 + lane;
        float pm = -INFINITY, pl = 0.0f;
        const bool mine = i < n && (i == 0 || p.head[2 * (c + i)].x);
        if (mine) {
          const float2 z = *reinterpret_cast<const float2*>(p.ml + 2 * at(i));
          pm = z.x;
          pl = z.y;
        }
        float top = fmaxf(pm, m);
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, s));
        const float ref = top == -INFINITY ? 0.0f : top;
        const float f0 = ex2(m - ref), f = ex2(pm - ref);
        float lsum = f * pl;
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) lsum += __shfl_xor_sync(0xffffffffu, lsum, s);
        l = l * f0 + lsum;
#pragma unroll
        for (int e = 0; e < V; ++e) o[e] *= f0;
        m = top;
        const uint32_t there = __ballot_sync(0xffffffffu, mine);
        const int left = min(32, n - i0);
        for (int s0 = 0; s0 < left; s0 += 8) {  // eight parts' loads in flight
          float y[8][V], w[8];
#pragma unroll
          for (int s = 0; s < 8; ++s) {
            w[s] = __shfl_sync(0xffffffffu, f, (s0 + s) & 31);
            const bool in = s0 + s < left && ((there >> (s0 + s)) & 1u);
#pragma unroll
            for (int e = 0; e < V; ++e) y[s][e] = 0.0f;
            if (in) load_part<V>(p.po + at(i0 + s0 + s) * D + lane * V, y[s]);
            if (!in) w[s] = 0.0f;
          }
#pragma unroll
          for (int s = 0; s < 8; ++s)
#pragma unroll
            for (int e = 0; e < V; ++e) o[e] = fmaf(w[s], y[s][e], o[e]);
        }
      }
    }
    const int64_t row = static_cast<int64_t>(open.y + tok) * p.H + j * p.G + hd;
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    uint32_t w[V / 2];
#pragma unroll
    for (int i = 0; i < V / 2; ++i) w[i] = bf16x2(o[2 * i] * inv, o[2 * i + 1] * inv);
    if constexpr (V == 4)
      *reinterpret_cast<uint2*>(p.out + row * D + lane * V) = make_uint2(w[0], w[1]);
    else
      *reinterpret_cast<uint32_t*>(p.out + row * D + lane * V) = w[0];
    if (p.lse && lane == 0) p.lse[row] = row_lse(m, l);
  }
}

int att_ctas() { return std::min(sm_count(), kMaxCtas); }

struct AttWs {
  size_t head, ml, po, total;
  explicit AttWs(int d) {
    const size_t n = static_cast<size_t>(att_ctas());
    size_t o = 0;
    head = o;  // (of 8 warps a CTA in the row kernel)
    o += (n * 16 * sizeof(int4) + 255) / 256 * 256;
    ml = o;
    o += n * 2 * kPartRows * 2 * sizeof(float);
    po = o;
    o += n * 2 * kPartRows * static_cast<size_t>(d) * sizeof(float);
    total = o;
  }
};

// The parameters that both kernels read, from the call's description.
inline AttParams att_params(const AttendLaunch& a, const DevCtl& ctl, int workers) {
  AttParams p{};
  p.Q = a.Q;
  p.kp = a.k_pages;
  p.vp = a.v_pages;
  p.bts = a.block_tables;
  p.cu_q = a.cu_q;
  p.lens = a.seq_lens;
  p.seq_of = a.seq_of;
  p.positions = a.positions;
  p.idx = a.idx;
  p.out = a.out;
  p.lse = a.lse;
  p.n_pages = a.n_pages;
  p.key_rows = a.n_pages << a.page_shift;
  p.max_blocks = a.max_blocks;
  p.page_shift = a.page_shift;
  p.n_seq = a.n_seq;
  p.n_tok = a.n_tok;
  p.H = a.H;
  p.Hkv = a.Hkv;
  p.G = a.H / a.Hkv;
  p.T = kTile / p.G;
  p.workers = workers;
  p.w_inv = workers > 1 ? ~uint64_t{0} / static_cast<uint64_t>(workers) + 1 : 0;
  p.g_inv = 65536 / p.G + 1;
  p.window = a.window;
  p.sinks = a.sinks;
  p.k = a.k;
  p.c = a.scale * 1.44269504088896340736f;
  p.ctl = ctl;
  const AttWs w(a.d);
  uint8_t* base = static_cast<uint8_t*>(a.ws);
  p.head = reinterpret_cast<int4*>(base + w.head);
  p.ml = reinterpret_cast<float*>(base + w.ml);
  p.po = reinterpret_cast<float*>(base + w.po);
  return p;
}

// The joining kernel, launched while the attention runs (it waits for its end
// before it reads).
template <int D>
cudaError_t launch_join(const AttParams& p, int part_rows, int y, cudaStream_t s) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(p.workers, y);
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, join_kernel<D>, p, part_rows);
}

}  // namespace

// The list form for few heads per key head (attend_rows.cu).
cudaError_t launch_attend_rows(const AttendLaunch& a, const DevCtl& ctl, cudaStream_t s);

}  // namespace misa
