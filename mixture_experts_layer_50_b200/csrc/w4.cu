// Products with 4-bit weights and group scales: the experts of a decode step.
//
//   out[r][i] = sum_c x[r][c] * (code(i, c) - 8) * scale(i, c / group)
//
// over the rows of every expert's group (and the shared expert's rows), with the SwiGLU or ReLU
// of an expert's first projection in the epilogue.
//
// Bound: HBM reads of the weights, half a byte each.  An SM has to take about 24 bytes, 49
// weights, per clock, so the cost per weight of turning codes into operands decides.  The
// matrices are stored in the order in which mma.sync reads its operand (include/moe.h): a lane's
// 16 bytes are four A fragments of m16n8k16, every 32-bit word one of them, whose codes two
// instructions turn into a register of two operands: (w >> 4i) & 0x000f000f | 0x4300 in each
// half is the bf16 number 128 + code, and subtracting 136 leaves code - 8, exactly.  The
// products with bf16 rows are exact in the fp32 accumulators; a group's sum is multiplied by
// its scale in fp32.  8-bit rows (e4m3 with scales) are widened to fp16, also exactly, and their
// scales join the weights' scales on the sums.  Nothing is rounded below 32 bits before the
// output.
//
// A warp owns 32 output rows (two blocks of 16; for SwiGLU a gate block and its up block) and
// all rows of one tile of a group: weights go from HBM to registers, kDepth steps of 128
// columns ahead, and straight into the tensor cores; the few activation rows come from L1.
// There is no barrier in the loop and none between warps unless the columns are split among
// the kSplit warps of an item, which small problems do to have enough loads in flight; the
// partial sums then meet in shared memory and are added in order.
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "common.cuh"
#include "kernels.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kDepth = 2;         // steps of 128 columns in flight per warp
constexpr int kMaxGroups = 1025;  // 1024 routed groups and the shared one

struct Args {
  const uint4* q;
  const uint32_t* scale;
  int rows, cols, parts, rb, ku, ng;
  const void* x;
  const float* x_scale;
  int xs_ld, xs_step;  // floats per row; 1: a scale per 128 columns, 0: one per row
  int64_t x_rows;
  const int32_t* row_index;
  const int32_t* offsets;
  int n_groups, has_shared;
  int64_t max_rows, shared_rows, shared_x_row0, shared_out_row0;
  int items_per_tile, split, act;
  float clamp;
  void* out;
  int out_f32;
  int* status;
};

__device__ __forceinline__ uint4 ldg_stream(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

template <bool kHalf>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                    uint32_t b1, bool zero) {
  const float c0 = zero ? 0.f : d[0], c1 = zero ? 0.f : d[1], c2 = zero ? 0.f : d[2],
              c3 = zero ? 0.f : d[3];
  if constexpr (kHalf)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c0), "f"(c1),
          "f"(c2), "f"(c3));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c0), "f"(c1),
          "f"(c2), "f"(c3));
}

// The four A registers of one word of codes.
template <bool kHalf>
__device__ __forceinline__ void widen(uint32_t w, uint32_t (&a)[4]) {
  if constexpr (kHalf) {
    // fp16 has room for a code at bits 4-7 too: 1024 + 16 code, brought back by * 1/16 - 72
    const __half2 k1032 = __floats2half2_rn(1032.f, 1032.f);
    const __half2 k16 = __floats2half2_rn(0.0625f, 0.0625f), k72 = __floats2half2_rn(-72.f, -72.f);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t v = i == 0 ? w : w >> 8;
      const uint32_t lo = (v & 0x000f000fu) | 0x64006400u, hi = (v & 0x00f000f0u) | 0x64006400u;
      const __half2 l = __hsub2(*reinterpret_cast<const __half2*>(&lo), k1032);
      const __half2 h = __hfma2(*reinterpret_cast<const __half2*>(&hi), k16, k72);
      a[2 * i] = *reinterpret_cast<const uint32_t*>(&l);
      a[2 * i + 1] = *reinterpret_cast<const uint32_t*>(&h);
    }
  } else {
    const __nv_bfloat162 k136 = __floats2bfloat162_rn(136.f, 136.f);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t v = ((w >> (4 * i)) & 0x000f000fu) | 0x43004300u;
      const __nv_bfloat162 r = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&v), k136);
      a[i] = *reinterpret_cast<const uint32_t*>(&r);
    }
  }
}

// Eight columns of a row as the B registers of two mma steps.
template <bool kX8>
__device__ __forceinline__ void load_x(const void* x, int64_t at, bool ok, uint32_t (&b)[4]) {
  if constexpr (kX8) {
    uint2 v = make_uint2(0, 0);
    if (ok) v = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(x) + at));
    const uint16_t p[4] = {(uint16_t)v.x, (uint16_t)(v.x >> 16), (uint16_t)v.y,
                           (uint16_t)(v.y >> 16)};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(b[i]) : "h"(p[i]));
  } else {
    uint4 v = make_uint4(0, 0, 0, 0);
    if (ok) v = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(x) + at));
    b[0] = v.x;
    b[1] = v.y;
    b[2] = v.z;
    b[3] = v.w;
  }
}

__device__ __forceinline__ float clip(float v, float c) { return v > c ? c : v < -c ? -c : v; }

template <int kNt, bool kX8, int kGroup>
__global__ void __launch_bounds__(kThreads, kNt == 4 ? 1 : 2) w4_kernel(const Args a) {
  constexpr int kTile = 8 * kNt;       // rows of a group that one item takes
  constexpr int kSteps = 128 / kGroup; // groups in 128 columns
  pdl_wait();
  __shared__ int32_t s_first[kMaxGroups + 1];  // first tile of each group
  __shared__ int32_t s_warp[kWarps];
  extern __shared__ float s_red[];  // [kWarps][8 kNt][32] when split
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int n_all = a.n_groups + a.has_shared;

  auto group_range = [&](int e, int64_t& first, int64_t& n) {
    if (e >= a.n_groups) {
      first = 0;
      n = a.shared_rows;
    } else if (a.offsets == nullptr) {
      first = 0;
      n = a.max_rows;
    } else {
      first = a.offsets[e];
      n = a.offsets[e + 1] - first;
      if (first < 0 || n < 0 || first + n > a.max_rows) n = -1;
    }
  };
  {
    // tiles of every group, and their exclusive scan
    const int per = (n_all + kThreads - 1) / kThreads;
    const int e0 = threadIdx.x * per;
    int mine = 0;
    bool bad = false;
    for (int e = e0; e < e0 + per && e < n_all; ++e) {
      int64_t first, n;
      group_range(e, first, n);
      if (n < 0) bad = true, n = 0;
      const int tiles = (int)((n + kTile - 1) / kTile);
      s_first[e] = tiles;
      mine += tiles;
    }
    if (bad && blockIdx.x == 0) report_status(a.status, kStatusInvalidInput);
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) s_warp[warp] = incl;
    __syncthreads();
    int at = incl - mine;
    for (int w = 0; w < warp; ++w) at += s_warp[w];
    for (int e = e0; e < e0 + per && e < n_all; ++e) {
      const int tiles = s_first[e];
      s_first[e] = at;
      at += tiles;
    }
    if (threadIdx.x == kThreads - 1) s_first[n_all] = at;
    __syncthreads();
  }
  const int64_t items = (int64_t)s_first[n_all] * a.items_per_tile;
  const int split = a.split, slots = kWarps / split;
  const int ks = warp % split;
  const int n_steps = (a.ku + 1) / 2;
  const int st0 = (int)((int64_t)n_steps * ks / split);
  const int st1 = (int)((int64_t)n_steps * (ks + 1) / split);

  for (int64_t it = (int64_t)blockIdx.x * slots; it < items; it += (int64_t)gridDim.x * slots) {
    const int64_t item = it + warp / split;
    const bool valid = item < items;
    float acc[2][kNt][4];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int n = 0; n < kNt; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[m][n][i] = 0.f;
    int e = 0, pair = 0, n_act = 0, tile_rows = 0;
    int64_t out_row0 = 0;
    if (valid) {
      const int tile = (int)(item / a.items_per_tile);
      pair = (int)(item % a.items_per_tile);
      int hi = n_all;  // the group that owns the tile: s_first[e] <= tile < s_first[e + 1]
      while (hi - e > 1) {
        const int mid = (e + hi) >> 1;
        if (s_first[mid] <= tile)
          e = mid;
        else
          hi = mid;
      }
      int64_t first, n;
      group_range(e, first, n);
      const int64_t row0 = (int64_t)(tile - s_first[e]) * kTile;
      tile_rows = (int)min((int64_t)kTile, n - row0);
      n_act = (tile_rows + 7) / 8;
      const bool shared = e >= a.n_groups;
      out_row0 = (shared ? a.shared_out_row0 : first) + row0;
      const int64_t in_row0 = (shared ? a.shared_x_row0 : first) + row0;

      // the input rows this lane reads, and those whose sums it holds
      int64_t x_at[kNt];
      int32_t xs_at[kNt][2];
      auto row_of = [&](int r) -> int64_t {
        if (r >= tile_rows) return -1;
        int64_t v = in_row0 + r;
        if (!shared && a.row_index != nullptr) v = a.row_index[v];
        if (v < 0 || v >= a.x_rows) {
          report_status(a.status, kStatusInvalidInput);
          return -1;
        }
        return v;
      };
#pragma unroll
      for (int n = 0; n < kNt; ++n) {
        const int64_t r = row_of(8 * n + g);
        x_at[n] = r < 0 ? -1 : r * a.cols;
        if (kX8) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int64_t rr = row_of(8 * n + 2 * t + i);
            xs_at[n][i] = rr < 0 ? -1 : (int32_t)rr;
          }
        }
      }
      // the item's two blocks of 16 rows
      int b0, b1;
      if (a.parts == 2) {
        b0 = pair;
        b1 = a.rb + pair;
      } else {
        b0 = 2 * pair;
        b1 = min(b0 + 1, a.rb - 1);
      }
      const int64_t blk = (int64_t)e * a.parts * a.rb;
      const uint4* q0 = a.q + (blk + b0) * a.ku * 32 + lane;
      const uint4* q1 = a.q + (blk + b1) * a.ku * 32 + lane;
      const uint32_t* sc0 = a.scale + (blk + b0) * a.ng * 8;
      const uint32_t* sc1 = a.scale + (blk + b1) * a.ng * 8;

      uint4 wq[kDepth][2][2];
      uint32_t ws[kDepth][2];
      auto fetch = [&](uint4 (&w)[2][2], uint32_t (&s)[2], int st) {
        const int u = 2 * st;
        const uint4 none = make_uint4(0x88888888u, 0x88888888u, 0x88888888u, 0x88888888u);
        w[0][0] = ldg_stream(q0 + (int64_t)u * 32);
        w[0][1] = ldg_stream(q1 + (int64_t)u * 32);
        if (u + 1 < a.ku) {
          w[1][0] = ldg_stream(q0 + (int64_t)(u + 1) * 32);
          w[1][1] = ldg_stream(q1 + (int64_t)(u + 1) * 32);
        } else {
          w[1][0] = w[1][1] = none;
        }
        // one word is the scales of rows g and g + 8; lane 8 i + j fetches word j of the i-th
        // group of the step (one group: every lane its own)
        const int gi = kSteps == 1 ? st : min(st * kSteps + (lane >> 3) % kSteps, a.ng - 1);
        const int wi = gi * 8 + (kSteps == 1 ? g : (lane & 7));
        s[0] = __ldg(sc0 + wi);
        s[1] = __ldg(sc1 + wi);
      };
#pragma unroll
      for (int p = 0; p < kDepth; ++p)
        if (st0 + p < st1) fetch(wq[p], ws[p], st0 + p);

      for (int s0 = st0; s0 < st1; s0 += kDepth) {
#pragma unroll
        for (int p = 0; p < kDepth; ++p) {
          const int st = s0 + p;
          if (st >= st1) break;
          uint4 w[2][2];
          uint32_t sw[2];
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            w[0][m] = wq[p][0][m];
            w[1][m] = wq[p][1][m];
            sw[m] = ws[p][m];
          }
          if (st + kDepth < st1) fetch(wq[p], ws[p], st + kDepth);
          float sx[kNt][2];
          if (kX8) {
#pragma unroll
            for (int n = 0; n < kNt; ++n)
#pragma unroll
              for (int i = 0; i < 2; ++i)
                sx[n][i] = xs_at[n][i] < 0 ? 0.f
                                           : __ldg(a.x_scale + (int64_t)xs_at[n][i] * a.xs_ld +
                                                   st * a.xs_step);
          }
          float part[2][kNt][4];
#pragma unroll
          for (int h = 0; h < 4; ++h) {
            const int col = 128 * st + 32 * h + 8 * t;
            uint32_t b[kNt][4];
#pragma unroll
            for (int n = 0; n < kNt; ++n)
              if (n < n_act) load_x<kX8>(a.x, x_at[n] + col, x_at[n] >= 0 && col < a.cols, b[n]);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
#pragma unroll
              for (int m = 0; m < 2; ++m) {
                const uint4& v = w[h >> 1][m];
                const uint32_t word = (h & 1) ? (j ? v.w : v.z) : (j ? v.y : v.x);
                uint32_t fa[4];
                widen<kX8>(word, fa);
#pragma unroll
                for (int n = 0; n < kNt; ++n)
                  if (n < n_act)
                    mma<kX8>(part[m][n], fa, b[n][2 * j], b[n][2 * j + 1],
                             j == 0 && h % (kGroup / 32) == 0);
              }
            }
            if ((h + 1) % (kGroup / 32) != 0) continue;
            const int gi = h / (kGroup / 32);
#pragma unroll
            for (int m = 0; m < 2; ++m) {
              const uint32_t s =
                  kSteps == 1 ? sw[m] : __shfl_sync(0xffffffffu, sw[m], gi * 8 + g);
              const float lo = __uint_as_float(s << 16), up = __uint_as_float(s & 0xffff0000u);
#pragma unroll
              for (int n = 0; n < kNt; ++n) {
                if (n >= n_act) continue;
                if (kX8) {
                  acc[m][n][0] = fmaf(part[m][n][0], lo * sx[n][0], acc[m][n][0]);
                  acc[m][n][1] = fmaf(part[m][n][1], lo * sx[n][1], acc[m][n][1]);
                  acc[m][n][2] = fmaf(part[m][n][2], up * sx[n][0], acc[m][n][2]);
                  acc[m][n][3] = fmaf(part[m][n][3], up * sx[n][1], acc[m][n][3]);
                } else {
                  acc[m][n][0] = fmaf(part[m][n][0], lo, acc[m][n][0]);
                  acc[m][n][1] = fmaf(part[m][n][1], lo, acc[m][n][1]);
                  acc[m][n][2] = fmaf(part[m][n][2], up, acc[m][n][2]);
                  acc[m][n][3] = fmaf(part[m][n][3], up, acc[m][n][3]);
                }
              }
            }
          }
        }
      }
    }
    if (split > 1) {
      __syncthreads();  // the previous item's sums have been read
      float* mine = s_red + (size_t)warp * (8 * kNt * 32) + lane;
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int n = 0; n < kNt; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) mine[((m * kNt + n) * 4 + i) * 32] = acc[m][n][i];
      __syncthreads();
      if (ks == 0) {
        for (int w = 1; w < split; ++w) {
          const float* other = mine + (size_t)w * (8 * kNt * 32);
#pragma unroll
          for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int n = 0; n < kNt; ++n)
#pragma unroll
              for (int i = 0; i < 4; ++i) acc[m][n][i] += other[((m * kNt + n) * 4 + i) * 32];
        }
      }
    }
    if (!valid || ks != 0) continue;
#pragma unroll
    for (int n = 0; n < kNt; ++n) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = 8 * n + 2 * t + (i & 1);
        if (r >= tile_rows) continue;
        const int64_t o = (out_row0 + r) * a.rows;
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          float v = acc[m][n][i];
          int b = pair;
          if (a.parts == 2) {
            if (m == 1) continue;
            float up = acc[1][n][i];
            if (a.clamp > 0.f) {
              v = clip(v, a.clamp);
              up = clip(up, a.clamp);
            }
            v = v / (1.f + expf(-v)) * up;
          } else {
            b = 2 * pair + m;
            if (a.act == 2) v = v < 0.f ? 0.f : v;
          }
          const int row = 16 * b + g + 8 * (i >> 1);
          if (row >= a.rows) continue;
          if (a.out_f32)
            static_cast<float*>(a.out)[o + row] = v;
          else
            static_cast<__nv_bfloat16*>(a.out)[o + row] = __float2bfloat16_rn(v);
        }
      }
    }
  }
}

template <int kNt, bool kX8>
cudaError_t launch_group(const Args& a, int group, int grid, size_t smem, cudaStream_t stream) {
  if (group == 32) return launch_pdl(w4_kernel<kNt, kX8, 32>, grid, kThreads, smem, stream, a);
  if (group == 64) return launch_pdl(w4_kernel<kNt, kX8, 64>, grid, kThreads, smem, stream, a);
  return launch_pdl(w4_kernel<kNt, kX8, 128>, grid, kThreads, smem, stream, a);
}

// One block turns 16 rows x 128 columns of bf16 weights into codes and scales.  A group's scale
// is its largest magnitude over 7, rounded to bf16 (stored as it is used); its codes are the
// quotients by that stored scale, rounded to the nearest whole number and kept in -8 .. 7.
__global__ void __launch_bounds__(256) w4_quantize_kernel(const __nv_bfloat16* __restrict__ w,
                                                          int rows, int cols, int rb, int ku,
                                                          int ng, int group, uint32_t* q,
                                                          __nv_bfloat16* scale) {
  pdl_wait();
  __shared__ float s_w[16][129];
  __shared__ float s_inv[16][4];
  const int steps = (ku + 1) / 2;
  const int st = blockIdx.x % steps;
  const int64_t blk = blockIdx.x / steps;  // (matrix and part, block of rows)
  const int b = (int)(blk % rb);
  const int64_t mat = blk / rb;
  for (int i = threadIdx.x; i < 16 * 128; i += 256) {
    const int r = i >> 7, c = i & 127, row = 16 * b + r, col = 128 * st + c;
    s_w[r][c] = row < rows && col < cols ? __bfloat162float(w[(mat * rows + row) * cols + col]) : 0.f;
  }
  __syncthreads();
  const int per = 128 / group;
  if (threadIdx.x < 16 * per) {
    const int r = threadIdx.x / per, gi = threadIdx.x % per;
    float m = 0.f;
    for (int c = 0; c < group; ++c) {
      const float v = fabsf(s_w[r][gi * group + c]);
      m = (v > m || v != v) ? v : m;  // a NaN stays
      if (m != m) break;
    }
    const __nv_bfloat16 s = __float2bfloat16_rn(m / 7.f);
    const int gg = st * per + gi;
    if (gg < ng) scale[((blk * ng + gg) * 8 + (r & 7)) * 2 + (r >> 3)] = s;
    const float f = __bfloat162float(s);
    s_inv[r][gi] = f == 0.f ? 0.f : f;
  }
  __syncthreads();
  const int u = threadIdx.x >> 7, lane = (threadIdx.x >> 2) & 31, word = threadIdx.x & 3;
  if (2 * st + u >= ku) return;
  uint32_t v = 0;
  for (int i = 0; i < 8; ++i) {
    const int e = i >> 2, p = (i >> 1) & 1, r = (i & 1) * 8 + (lane >> 2);
    const int c = 64 * u + 32 * (word >> 1) + 8 * (lane & 3) + 4 * (word & 1) + 2 * p + e;
    const float f = s_inv[r][c / group];
    const float x = f == 0.f ? 0.f : rintf(s_w[r][c] / f);
    const int code = (int)fminf(fmaxf(x, -8.f), 7.f) + 8;
    v |= (uint32_t)code << (4 * i);
  }
  q[((blk * ku + 2 * st + u) * 32 + lane) * 4 + word] = v;
}

}  // namespace

cudaError_t launch_w4_quantize(const void* w, int64_t mats, int rows, int cols, int group, void* q,
                               void* scale, cudaStream_t stream, int* launches) {
  const int rb = (rows + 15) / 16, ku = (cols + 63) / 64, ng = (cols + group - 1) / group;
  const int64_t blocks = mats * rb * ((ku + 1) / 2);
  ++*launches;
  return launch_pdl(w4_quantize_kernel, (unsigned)blocks, 256, 0, stream,
                    static_cast<const __nv_bfloat16*>(w), rows, cols, rb, ku, ng, group,
                    static_cast<uint32_t*>(q), static_cast<__nv_bfloat16*>(scale));
}

cudaError_t launch_w4(const W4Gemm& p, cudaStream_t stream, int* launches) {
  Args a{};
  a.q = static_cast<const uint4*>(p.q);
  a.scale = static_cast<const uint32_t*>(p.scale);
  a.rows = p.rows;
  a.cols = p.cols;
  a.parts = p.parts;
  a.rb = (p.rows + 15) / 16;
  a.ku = (p.cols + 63) / 64;
  a.ng = (p.cols + p.group - 1) / p.group;
  a.x = p.x;
  a.x_scale = p.x_scale;
  a.xs_step = p.x_group != 0;
  a.xs_ld = p.x_group != 0 ? (p.cols + 127) / 128 : 1;
  a.x_rows = p.x_rows;
  a.row_index = p.row_index;
  a.offsets = p.offsets;
  a.n_groups = p.n_groups;
  a.has_shared = p.has_shared;
  a.max_rows = p.max_rows;
  a.shared_rows = p.shared_rows;
  a.shared_x_row0 = p.shared_x_row0;
  a.shared_out_row0 = p.shared_out_row0;
  a.items_per_tile = p.parts == 2 ? a.rb : (a.rb + 1) / 2;
  a.act = p.relu ? 2 : 0;
  a.clamp = p.clamp;
  a.out = p.out;
  a.out_f32 = p.out_f32;
  a.status = p.status;
  // rows of a tile: enough for the largest group there can be, 32 at most
  const int64_t most = p.has_shared ? (p.shared_rows > p.max_group_rows ? p.shared_rows : p.max_group_rows)
                                    : p.max_group_rows;
  const int nt = most <= 8 ? 1 : most <= 16 ? 2 : 4;
  // split the columns among warps until there are about 16 warps' loads in flight on each SM,
  // four steps or more to a warp
  const int sms = tc::num_sms();
  const int64_t groups = (p.max_rows < p.n_groups ? p.max_rows : p.n_groups) + p.has_shared;
  const int64_t items = groups * a.items_per_tile;
  a.split = 1;
  while (a.split < kWarps && items * a.split < 16 * sms && (a.ku + 1) / 2 >= 8 * a.split)
    a.split *= 2;
  const int64_t tile = 8 * nt;
  const int64_t tiles = p.max_rows / tile + (p.max_rows < p.n_groups ? p.max_rows : p.n_groups) +
                        (p.has_shared ? (p.shared_rows + tile - 1) / tile : 0);
  const int64_t blocks = (tiles * a.items_per_tile * a.split + kWarps - 1) / kWarps;
  const int64_t full = (nt == 4 ? 1 : 2) * (int64_t)sms;
  const int grid = (int)(blocks < 1 ? 1 : blocks < full ? blocks : full);
  const size_t smem = a.split > 1 ? sizeof(float) * kWarps * 8 * nt * 32 : 0;
  ++*launches;
  if (p.x_scale != nullptr)
    return nt == 1   ? launch_group<1, true>(a, p.group, grid, smem, stream)
           : nt == 2 ? launch_group<2, true>(a, p.group, grid, smem, stream)
                     : launch_group<4, true>(a, p.group, grid, smem, stream);
  return nt == 1   ? launch_group<1, false>(a, p.group, grid, smem, stream)
         : nt == 2 ? launch_group<2, false>(a, p.group, grid, smem, stream)
                   : launch_group<4, false>(a, p.group, grid, smem, stream);
}

}  // namespace moe
