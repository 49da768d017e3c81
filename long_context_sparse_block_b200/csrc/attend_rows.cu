// Attention over selected tokens for at most 16 query heads per key head.
//
// The same sums as attend.cu's list form (o = sum over the list of softmax
// weights times values, one pass with a running reference).  With few heads per
// gathered row the work is the gather: 4 D bytes per listed token and key head
// against 4 D G flops, read from L2 as the lists of many rows overlap.  A
// 128-row tcgen05 tile would hold G live rows, and its long per-tile chain (one
// live warp of four) takes 2 us for 128 tokens; here a warp owns a (row, key
// head) unit by itself, m16n8k16 products with the G heads as the 16 rows, and
// eight such warps on an SM hide each other's latencies.  (1055 rows of 333
// tokens, 24 heads of 64 over 4 key heads: 173 us with the tcgen05 tile.)
//
// A warp keeps a ring of entries in shared memory, each the key rows or the
// value rows of 32 tokens, filled by cp.async with the lanes of a row's 16-byte
// units side by side; it copies ahead over the units' ends, token ids two groups
// and table entries one group ahead of the copies.  No warp waits for another.
// The units' groups are laid on a line that is cut evenly over all warps; parts
// are joined as in attend.cu.
#include <atomic>

#include "attend.cuh"

namespace misa {
namespace {

constexpr int kWarps = 8;
constexpr int kGroup = 32;  // tokens of a ring entry
constexpr int kRows = 16;

template <int D>
struct RowLayout {
  static constexpr int ENTRY = kGroup * D * 2;
  static constexpr int ENTRIES = D == 128 ? 3 : 6;
  static constexpr int MASKS = 8;  // words of visible tokens, by group
  static constexpr int WARP_BYTES = ENTRIES * ENTRY;
  static constexpr int OFF_MASK = kWarps * WARP_BYTES;
  static constexpr int BYTES = OFF_MASK + kWarps * MASKS * 4;
};

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&v)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_trans(uint32_t addr, uint32_t (&v)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
               : "r"(addr)
               : "memory");
}
// c += a b, a [16 x 16], b [16 x 8], bf16 with fp32 sums.
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
      "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// A stretch of the line of groups: token t, key head j, group i of nt, `left` more.
struct Cursor {
  int t, j, i;
  int64_t left;
  __device__ __forceinline__ void step(const AttParams& p, int nt) {
    --left;
    if (++i == nt) {
      i = 0;
      if (++j == p.Hkv) {
        j = 0;
        ++t;
      }
    }
  }
};

template <int D>
__global__ void __launch_bounds__(kWarps * 32, 1) list_rows_kernel(const AttParams p) {
  using L = RowLayout<D>;
  constexpr int E = L::ENTRIES, UPR = D / 8;
  extern __shared__ __align__(128) uint8_t smem_rows[];
  const int lane = lane_id();
  const int worker = warp_id() * gridDim.x + blockIdx.x;  // few workers: one per SM first
  const uint32_t ring = smem_u32(smem_rows) + warp_id() * L::WARP_BYTES;
  volatile uint32_t* masks =
      reinterpret_cast<volatile uint32_t*>(smem_rows + L::OFF_MASK) + warp_id() * L::MASKS;
  asm volatile("griddepcontrol.launch_dependents;");  // the joining kernel may get ready

  const int nt = (p.k + kGroup - 1) / kGroup;
  Cursor cur;
  {
    const int64_t total = static_cast<int64_t>(p.n_tok) * p.Hkv * nt;
    const int64_t x0 = cut(p, p.workers, total, min(worker, p.workers));
    const int64_t x1 = cut(p, p.workers, total, min(worker + 1, p.workers));
    const int64_t unit = x0 / nt;
    cur.t = static_cast<int>(unit / p.Hkv);
    cur.j = static_cast<int>(unit % p.Hkv);
    cur.i = static_cast<int>(x0 % nt);
    cur.left = x1 - x0;
    if (lane == 0 && worker < p.workers) {
      int4 cont = make_int4(0, 0, 0, 0), open = make_int4(0, 0, 0, 0);
      cont.x = cur.i > 0 && cur.left > 0;
      const int64_t ue = x1 / nt;
      if (x1 % nt != 0 && x1 > x0 && ue * nt >= x0) {
        const int t = static_cast<int>(ue / p.Hkv);
        const int b = __ldg(p.seq_of + t);
        if (b >= 0 && b < p.n_seq)  // (else: left as it was)
          open = make_int4(1, t, 1 | static_cast<int>(ue - static_cast<int64_t>(t) * p.Hkv) << 16,
                           last_worker(p, p.workers, total, (ue + 1) * nt));
      }
      p.head[2 * worker] = cont;
      p.head[2 * worker + 1] = open;
    }
  }

  // ---- copies ahead.  A group passes three steps: token ids (a), table entries
  // (b), copies (c); `ahead` is the next group whose ids are read.
  const int64_t cap = static_cast<int64_t>(p.max_blocks) << p.page_shift;
  struct Ahead {
    int s, pg, pos, j, live;
    const int32_t* bt;
  };
  Cursor ahead = cur;
  auto read_ids = [&](Ahead& a) {
    a.live = 0;
    a.s = -1;
    a.pos = -1;
    a.j = 0;
    a.bt = p.bts;
    if (ahead.left <= 0) return;
    const int b = __ldg(p.seq_of + ahead.t);
    if (b >= 0 && b < p.n_seq) {
      const int e = ahead.i * kGroup + lane;
      if (e < p.k) a.s = __ldg(p.idx + static_cast<int64_t>(ahead.t) * p.k + e);
      a.pos = __ldg(p.positions + ahead.t);
      a.bt = p.bts + static_cast<int64_t>(b) * p.max_blocks;
    } else if (b >= p.n_seq) {
      report(p.ctl, DEV_BAD_INPUT);
    }
    a.j = ahead.j;
    a.live = 1;
    ahead.step(p, nt);
  };
  auto read_page = [&](Ahead& a) {
    a.pg = a.s >= 0 && a.s <= a.pos && a.s < cap ? __ldg(a.bt + (a.s >> p.page_shift)) : 0;
  };
  Ahead a0, a1, a2;  // copies next, table entry read, ids read
  read_ids(a0);
  read_page(a0);
  read_ids(a1);
  read_page(a1);
  read_ids(a2);
  int row = -1, head = 0, more = 0;  // cache row of this lane's token of the group being copied
  uint32_t copied = 0;               // entries copied so far
  // Copies the next entry (key rows, then value rows, of the next group).
  auto copy_next = [&]() {
    const bool keys = (copied & 1) == 0;
    if (keys) {
      row = -1;
      more = a0.live;
      head = a0.j;
      if (a0.s >= 0 && a0.s <= a0.pos) {
        int pg = a0.pg;
        if (a0.s >= cap) {
          report(p.ctl, DEV_BAD_INPUT);
        } else {
          if (pg < 0 || pg >= p.n_pages) {
            report(p.ctl, DEV_BAD_INPUT);
            pg = 0;
          }
          row = (pg << p.page_shift) | (a0.s & ((1 << p.page_shift) - 1));
        }
      }
      const uint32_t seen = __ballot_sync(0xffffffffu, row >= 0);
      if (lane == 0) masks[(copied >> 1) % L::MASKS] = seen;
      a0 = a1;
      a1 = a2;
      read_page(a1);
      read_ids(a2);
    }
    if (more) {
      const uint32_t dst = ring + (copied % E) * L::ENTRY;
      const uint16_t* base = (keys ? p.kp : p.vp) + head * D + (lane % UPR) * 8;
#pragma unroll
      for (int i = 0; i < UPR; ++i) {
        const int r = i * (32 / UPR) + lane / UPR;
        const int y = __shfl_sync(0xffffffffu, row, r);
        cp_async16(dst + r * (D * 2) + (((lane % UPR) ^ (r & 7)) << 4),
                   base + static_cast<int64_t>(y < 0 ? 0 : y) * p.Hkv * D, y < 0 ? 0u : 16u);
      }
    }
    cp_async_commit();
    ++copied;
  };
#pragma unroll
  for (int i = 0; i < E; ++i) copy_next();

  // ---- sums.  Lane: rows (heads) g and g + 8; columns 2 c, 2 c + 1 of each eight.
  const int g = lane >> 2, c = lane & 3;
  uint32_t q[D / 16][4];
  float o[D / 8][4];
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
  uint32_t done = 0;  // groups summed
  int start = cur.i;  // first group of the segment
  bool fresh = true, live = false;
  while (cur.left > 0) {
    if (fresh) {
      const int b = __ldg(p.seq_of + cur.t);
      live = b >= 0 && b < p.n_seq;
      const uint16_t* qr = p.Q + (static_cast<int64_t>(cur.t) * p.H + cur.j * p.G) * D + 2 * c;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int r = g + 8 * (x & 1);
          q[kk][x] = live && r < p.G
                         ? __ldg(reinterpret_cast<const uint32_t*>(qr + r * D + kk * 16 + 8 * (x >> 1)))
                         : 0u;
        }
#pragma unroll
      for (int x = 0; x < D / 8; ++x)
#pragma unroll
        for (int y = 0; y < 4; ++y) o[x][y] = 0.0f;
      m[0] = m[1] = -INFINITY;
      l[0] = l[1] = 0.0f;
      start = cur.i;
      fresh = false;
    }
    const uint32_t ek = 2 * done;
    cp_async_wait_group<E - 1>();
    __syncwarp();
    const uint32_t seen = masks[done % L::MASKS];
    if (seen) {
      // S: 16 heads x 32 tokens
      float s[4][4];
      const uint32_t kb = ring + (ek % E) * L::ENTRY;
#pragma unroll
      for (int x = 0; x < 4; ++x)
#pragma unroll
        for (int y = 0; y < 4; ++y) s[x][y] = 0.0f;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
        for (int x = 0; x < 2; ++x) {  // 16 tokens: matrices (tokens 0-7, 8-15) x (k 0-7, 8-15)
          const int r = x * 16 + (lane & 7) + ((lane >> 3) & 1) * 8, u = kk * 2 + (lane >> 4);
          uint32_t b[4];
          ldsm4(kb + r * (D * 2) + ((u ^ (r & 7)) << 4), b);
          mma16816(s[2 * x], q[kk], b[0], b[2]);
          mma16816(s[2 * x + 1], q[kk], b[1], b[3]);
        }
      __syncwarp();
      copy_next();
      if (seen != 0xffffffffu) {
#pragma unroll
        for (int x = 0; x < 4; ++x)
#pragma unroll
          for (int y = 0; y < 4; ++y)
            if (!((seen >> (x * 8 + 2 * c + (y & 1))) & 1u)) s[x][y] = -INFINITY;
      }
      uint32_t pa[2][4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {  // rows g, g + 8
        float top = -INFINITY;
#pragma unroll
        for (int x = 0; x < 4; ++x) top = fmaxf(top, fmaxf(s[x][2 * h], s[x][2 * h + 1]));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2)) * p.c;
        const bool raise = top > m[h] + (m[h] == -INFINITY ? 0.0f : kRaise);
        if (__any_sync(0xffffffffu, raise)) {
          const float mn = raise ? top : m[h];
          const float f = raise ? ex2(m[h] - mn) : 1.0f;
          m[h] = mn;
          l[h] *= f;
#pragma unroll
          for (int x = 0; x < D / 8; ++x) {
            o[x][2 * h] *= f;
            o[x][2 * h + 1] *= f;
          }
        }
        const float ref = m[h] == -INFINITY ? 0.0f : m[h];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const float e0 = ex2(fmaf(s[x][2 * h], p.c, -ref)), e1 = ex2(fmaf(s[x][2 * h + 1], p.c, -ref));
          l[h] += e0 + e1;
          pa[x >> 1][h + 2 * (x & 1)] = bf16x2(e0, e1);
        }
      }
      cp_async_wait_group<E - 1>();
      __syncwarp();
      const uint32_t vb = ring + ((ek + 1) % E) * L::ENTRY;
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int d = 0; d < D / 16; ++d) {  // 16 columns: matrices (tokens 0-7, 8-15) x (8, 8)
          const int r = x * 16 + (lane & 15), u = d * 2 + (lane >> 4);
          uint32_t b[4];
          ldsm4_trans(vb + r * (D * 2) + ((u ^ (r & 7)) << 4), b);
          mma16816(o[2 * d], pa[x], b[0], b[1]);
          mma16816(o[2 * d + 1], pa[x], b[2], b[3]);
        }
      __syncwarp();
      copy_next();
    } else {  // nothing visible among these tokens
      copy_next();
      cp_async_wait_group<E - 1>();
      __syncwarp();
      copy_next();
    }
    ++done;
    const int i = cur.i, t = cur.t, j = cur.j;
    cur.step(p, nt);
    if (i + 1 < nt && cur.left > 0) continue;

    // ---- the segment's result
    fresh = true;
    if (!live) continue;  // a row of no sequence: left as it was
    const int part = start > 0 ? 2 * worker : i + 1 < nt ? 2 * worker + 1 : -1;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float sum = l[h];
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
      const int r = g + 8 * h;
      if (r >= p.G) continue;
      if (part >= 0) {
        const int64_t at = static_cast<int64_t>(part) * kRows + r;
        if (c == 0) *reinterpret_cast<float2*>(p.ml + 2 * at) = make_float2(m[h], sum);
#pragma unroll
        for (int x = 0; x < D / 8; ++x)
          *reinterpret_cast<float2*>(p.po + at * D + x * 8 + 2 * c) =
              make_float2(o[x][2 * h], o[x][2 * h + 1]);
      } else {
        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
        const int64_t at = static_cast<int64_t>(t) * p.H + j * p.G + r;
#pragma unroll
        for (int x = 0; x < D / 8; ++x)
          *reinterpret_cast<uint32_t*>(p.out + at * D + x * 8 + 2 * c) =
              bf16x2(o[x][2 * h] * inv, o[x][2 * h + 1] * inv);
        if (p.lse && c == 0) p.lse[at] = row_lse(m[h], sum);
      }
    }
  }
  cp_async_wait_all();
}

template <int D>
cudaError_t launch_rows(const AttParams& p, cudaStream_t s) {
  using L = RowLayout<D>;
  static std::atomic<uint64_t> ready{0};  // devices whose shared-memory limit is raised
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !(ready.load() >> dev & 1)) {
    e = cudaFuncSetAttribute(list_rows_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::BYTES);
    if (e != cudaSuccess) return e;
    if (dev < 64) ready.fetch_or(uint64_t{1} << dev);
  }
  const int n = att_ctas();
  list_rows_kernel<D><<<n, kWarps * 32, L::BYTES, s>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess || p.workers == 1) return e;
  return launch_join<D>(p, kRows, 1, s);
}

}  // namespace

cudaError_t launch_attend_rows(const AttendLaunch& a, const DevCtl& ctl, cudaStream_t s) {
  // at least 4 groups a worker: below that a unit falls into so many parts that
  // joining them costs more than the shorter stretches save (8 rows of 2048 tokens,
  // 16 heads: 47 us with one group a worker, 18 us with four)
  const int64_t groups =
      static_cast<int64_t>(a.n_tok) * a.Hkv * ((a.k + kGroup - 1) / kGroup);
  const int workers =
      static_cast<int>(std::min<int64_t>(att_ctas() * kWarps, std::max<int64_t>(1, groups / 4)));
  const AttParams p = att_params(a, ctl, workers);
  return a.d == 128 ? launch_rows<128>(p, s) : launch_rows<64>(p, s);
}

}  // namespace misa
