// What the attention kernels share: the launch's parameters, the units of work of
// a packed batch, the workspace of units that were cut into parts and the kernel
// that joins them.
#pragma once

#include <algorithm>

#include "internal.h"

namespace misa {
namespace {

constexpr int kTile = 128;       // keys per tile of the dense form
constexpr int kBlockRows = 256;  // rows of a unit (two slots of 128)
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
  int g_inv;                // 65536 / G + 1: x / G == x * g_inv >> 16 for x < 384, G <= 128
  int window;               // 0: none
  int sinks;
  int k;
  float c;                  // scale * log2(e)
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

__device__ __forceinline__ int64_t row_blocks(const AttParams& p, const SeqInfo& s) {
  return (static_cast<int64_t>(s.n) * p.G + kBlockRows - 1) / kBlockRows;
}

// Cost of row block m of a sequence and its sum over blocks 0..m-1: about the
// keys it passes over, times G.  Only the balance depends on it.
__device__ __forceinline__ int64_t cost_flat(const AttParams& p) {
  return p.window ? static_cast<int64_t>(p.G) * (static_cast<int64_t>(p.window) + p.sinks + 2 * kTile) +
                        kBlockRows
                  : 0x3fffffffffffffffLL;
}
__device__ __forceinline__ int64_t cost_of(const AttParams& p, const SeqInfo& s, int64_t m) {
  const int64_t c = static_cast<int64_t>(p.G) * (max(s.p0, 0) + kTile) + kBlockRows * (m + 1);
  return min(c, cost_flat(p));
}
__device__ __forceinline__ int64_t cost_before(const AttParams& p, const SeqInfo& s, int64_t m) {
  const int64_t base = static_cast<int64_t>(p.G) * (max(s.p0, 0) + kTile);
  const int64_t flat = cost_flat(p);
  // blocks below `lin` grow with m, those from it on cost `flat`
  int64_t lin = flat > base ? (flat - base) / kBlockRows : 0;
  lin = min(lin, m);
  return lin * base + kBlockRows * (lin * (lin + 1) / 2) + (m - lin) * (m > lin ? flat : 0);
}

// Tiles of a unit: `sink` tiles from the start, then tiles lo.. .
struct Tiles {
  int n;     // tiles in all
  int sink;
  int lo;
  int rows;  // valid rows of the unit
};

__device__ __forceinline__ Tiles unit_tiles(const AttParams& p, const SeqInfo& s, int m) {
  Tiles t;
  const int64_t r0 = static_cast<int64_t>(m) * kBlockRows;
  const int64_t all = static_cast<int64_t>(s.n) * p.G;
  t.rows = static_cast<int>(min(static_cast<int64_t>(kBlockRows), all - r0));
  const int p_first = s.p0 + static_cast<int>(r0 / p.G);
  const int p_last = s.p0 + static_cast<int>((r0 + t.rows - 1) / p.G);
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
// Joins the parts of the unit that worker blockIdx.x (a CTA, or a warp of the row
// kernel) opened and did not finish:
//   o = sum_i 2^(m_i - m) o_i / sum_i 2^(m_i - m) l_i,  parts in worker order.
// A warp takes a row: its lanes hold the parts' m and l, 32 at a time.  What it
// finds in head[2 w] and head[2 w + 1] of worker w:
//   head[2 w]     x: 1 if w has a part of a unit that an earlier worker opened, in
//                 slot 2 w, y: 1 if that unit ends there
//   head[2 w + 1] x: 1 if w opens a unit that it does not finish (slot 2 w + 1),
//                 y: sequence (list form: 0), z: row block (token), w: key head
constexpr int kJoinThreads = 256;
constexpr int kJoinRows = 8;       // rows of a block at a time
constexpr int kMaxParts = 520;     // of one unit: 16384 listed tokens by 32, and the ends

template <int D, bool LIST>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const AttParams p, int workers, int part_rows) {
  __shared__ int parts[kMaxParts];  // workspace slots of the unit's parts, in order
  __shared__ int first_end, warp_n[kJoinThreads / 32];
  const int c = blockIdx.x;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the attention kernel is done
  const int4 open = p.head[2 * c + 1];
  if (!open.x) return;
  int64_t t0;
  int rows;
  if constexpr (LIST) {
    if (open.z >= p.n_tok) return;
    const int b = __ldg(p.seq_of + open.z);
    if (b < 0 || b >= p.n_seq) return;
    t0 = open.z;
    rows = p.G;
  } else {
    const SeqInfo s = seq_info(p, open.y);
    const Tiles t = unit_tiles(p, s, open.z);
    t0 = s.t0;
    rows = t.rows;
  }
  if (static_cast<int>(blockIdx.y) * 8 >= rows) return;
  // the workers that follow, up to the one that ends the unit (one whose share of
  // it is less than a tile has no part)
  int n = 1;
  if (threadIdx.x == 0) {
    parts[0] = 2 * c + 1;
    first_end = workers;
  }
  for (int e0 = c + 1; e0 < workers; e0 += kJoinThreads) {
    const int e = e0 + static_cast<int>(threadIdx.x);
    const int4 cont = e < workers ? p.head[2 * e] : make_int4(0, 0, 0, 0);
    __syncthreads();
    if (cont.y) atomicMin(&first_end, e);
    __syncthreads();
    const int end = first_end;
    const bool mine = cont.x && e <= end;
    const uint32_t vote = __ballot_sync(0xffffffffu, mine);
    if (lane_id() == 0) warp_n[warp_id()] = __popc(vote);
    __syncthreads();
    int at = n;
    for (int w = 0; w < kJoinThreads / 32; ++w) {
      if (w < warp_id()) at += warp_n[w];
      n += warp_n[w];
    }
    at += __popc(vote & ((1u << lane_id()) - 1u));
    if (mine && at < kMaxParts) parts[at] = 2 * e;
    if (end < e0 + kJoinThreads) break;
  }
  n = min(n, kMaxParts);
  __syncthreads();

  constexpr int V = D / 32;  // elements of a lane
  const int lane = lane_id();
  for (int r = blockIdx.y * 8 + warp_id(); r < rows; r += gridDim.y * 8) {
    float m = -INFINITY, l = 0.0f, o[V];
#pragma unroll
    for (int i = 0; i < V; ++i) o[i] = 0.0f;
    for (int i0 = 0; i0 < n; i0 += 32) {
      float pm = -INFINITY, pl = 0.0f;
      int64_t q = 0;
      if (i0 + lane < n) {
        q = static_cast<int64_t>(parts[i0 + lane]) * part_rows + r;
        const float2 x = *reinterpret_cast<const float2*>(p.ml + 2 * q);
        pm = x.x;
        pl = x.y;
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
      for (int i = 0; i < V; ++i) o[i] *= f0;
      m = top;
      const int left = min(32, n - i0);
#pragma unroll 4
      for (int x = 0; x < left; ++x) {
        const float w = __shfl_sync(0xffffffffu, f, x);
        const int64_t qx = __shfl_sync(0xffffffffu, q, x);
        float y[V];
        if constexpr (V == 4) {
          const float4 z = *reinterpret_cast<const float4*>(p.po + qx * D + lane * V);
          y[0] = z.x, y[1] = z.y, y[2] = z.z, y[3] = z.w;
        } else {
          const float2 z = *reinterpret_cast<const float2*>(p.po + qx * D + lane * V);
          y[0] = z.x, y[1] = z.y;
        }
#pragma unroll
        for (int i = 0; i < V; ++i) o[i] = fmaf(w, y[i], o[i]);
      }
    }
    const int64_t rr = (LIST ? 0 : static_cast<int64_t>(open.z) * kBlockRows) + r;
    const int64_t row = (t0 + rr / p.G) * p.H + open.w * p.G + rr % p.G;
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    uint32_t w[V / 2];
#pragma unroll
    for (int i = 0; i < V / 2; ++i) w[i] = bf16x2(o[2 * i] * inv, o[2 * i + 1] * inv);
    if constexpr (V == 4)
      *reinterpret_cast<uint2*>(p.out + row * D + lane * V) = make_uint2(w[0], w[1]);
    else
      *reinterpret_cast<uint32_t*>(p.out + row * D + lane * V) = w[0];
    if (p.lse && lane == 0)
      p.lse[row] = row_lse(m, l);
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
    o += n * 2 * kBlockRows * 2 * sizeof(float);
    po = o;
    o += n * 2 * kBlockRows * static_cast<size_t>(d) * sizeof(float);
    total = o;
  }
};

// The parameters that both kernels read, from the call's description.
inline AttParams att_params(const AttendLaunch& a, const DevCtl& ctl) {
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
template <int D, bool LIST>
cudaError_t launch_join(const AttParams& p, int workers, int part_rows, int y, cudaStream_t s) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(workers, y);
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, join_kernel<D, LIST>, p, workers, part_rows);
}

}  // namespace

// The list form for few heads per key head (attend_rows.cu).
cudaError_t launch_attend_rows(const AttendLaunch& a, const DevCtl& ctl, cudaStream_t s);

}  // namespace misa
