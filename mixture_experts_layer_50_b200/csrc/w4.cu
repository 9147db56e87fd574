// Products with 4-bit weights and group scales: the experts of a decode step.
//
//   out[r][i] = sum_c x[r][c] * (code(i, c) - 8) * scale(i, c / group)
//
// over the rows of every expert's group (and the shared expert's rows), with the SwiGLU or ReLU
// of an expert's first projection in the epilogue.
//
// Bound: HBM reads of the weights, half a byte each.  An SM has to take about 24 bytes, 49
// weights, per clock, so the instructions that turn codes into operands decide.  The matrices are
// stored in the order in which mma.sync reads its operand (include/moe.h): a lane's 16 bytes are
// four A fragments of m16n8k16, every 32-bit word one of them, and masks alone make operands of
// it.  Bits in the low byte of a 16-bit float, all else zero, are the number bits * 2^-133 in bf16
// (subnormal up to 127, and on evenly from there: the mantissa has seven bits), bits * 2^-24 in
// fp16.  A byte holds the codes of rows g and g + 8; so w & 0x00ff00ff gives code(g) + 16
// code(g + 8), w & 0x000f000f code(g) alone, and one byte permutation and one mask the same for
// the word's other columns: four instructions for eight weights.  The fragment's rows g take the
// first, its rows g + 8 the second, and the difference of their sums is 16 times the sum of row
// g + 8.  The 8 that every code is too large by is -8 sum(x) over a group of columns, the same for
// all weights: it is made once, where the rows arrive, and is what the group's sums start from.
// The powers of two go into the result at the end.  To keep bf16 products out of fp32's own
// subnormal range, the rows are multiplied by 2^65 as they arrive in shared memory; so a row's
// numbers count as infinite from 2^63 on.  8-bit rows (e4m3 with scales) become fp16 there, and
// their scales join the weights' scales on the sums.  All products are exact in the fp32
// accumulators; a group's sum is multiplied by its scale in fp32, and nothing is rounded below 32
// bits before the output.  (For one token at 4096 x 14336 x 2: 33 us with a subtraction for each
// operand, 17.3 us with five instructions for a word, 16.2 us with four.  mma.sync takes the
// operands from the registers that they are made in and is 20 to 32 % busy.  The fifth-generation
// tensor cores take them from shared or tensor memory, so each decoded weight would be stored
// first, at 16 bits; in return one decoding could serve all rows of a group, which here every tile
// of 16 rows does again.  Not built: at up to 16 rows there is nothing to share.)
//
// A block of 16 warps, one on an SM, owns one tile of a group's rows (8 or 16) and 512 output
// rows, each warp two blocks of 16 of them (for SwiGLU a gate block and its up block).  Every warp
// runs a ring of its own in shared memory for the weights that it alone needs: each lane copies
// asynchronously what that lane will read, kDepth steps of 256 columns ahead and on across items,
// without a barrier (registers held no more than two steps of 128, and waited for one another).
// 16 warps leave each thread 128 registers; tiles of 16 rows spill 16 to 80 bytes of them.
// The activation rows, which all warps need, come in chunks of several steps into three buffers:
// every warp copies its part of a chunk two chunks ahead and makes operands of it one chunk ahead,
// and mbarriers tell when all have, so the warps may run apart by most of a chunk.
//
// The items are dealt to the resident blocks in whole rounds, there and back, those of more than 8
// rows first: they take nearly twice as long as the others, and so meet the cheapest at the end (37
// tokens on 48 experts and a shared one: 224 us, 269 us in the groups' order).  Those that are
// left, or all where there are few, are cut into 2, 4, 8 or 16 units, whose warps share out the
// columns of fewer output rows; their partial sums meet in shared memory and are added in order.
// Where items are few and their rows take the room that a cut needs, clusters of 2 to 8 blocks share
// out the columns instead, and the first adds the others' sums in order (33 8-bit rows of 14336
// columns: 204 us without, 61 us in clusters of 4, 55 us of 6).
#include <cooperative_groups.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <climits>

#include <atomic>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "mbar.cuh"

namespace moe {
namespace {

namespace cg = cooperative_groups;

struct Args {
  const uint4* q;
  const uint32_t* scale;
  int rows, cols, parts, rb, ku, ng;
  const void* x;
  const float* x_scale;
  int xs_ld, xs_step;  // floats per row; 1: a scale per 128 columns, 0: one per row
  int x_rows;
  const int32_t* row_index;
  const int32_t* offsets;
  int n_groups, has_shared;
  int max_rows, max_group_rows, shared_rows, shared_x_row0, shared_out_row0;
  int pairs, max_split, x_steps, buf_bytes, tables, cluster, relu;
  float clamp;
  void* out;
  int out_f32;
  int* status;
  int give_up;  // self-test: a warp of the grid that starts as if a wait had run out, or -1
};

// Warps of a block, as many as the registers allow (one block on an SM), and the steps of 256
// columns in a warp's ring, of two blocks' weights and scales each.
constexpr int kWarps = 16, kThreads = 32 * kWarps, kDepth = 2;
constexpr int kDynamicSmem = 226 * 1024;  // of 227 KB, less the barriers and small tables
constexpr int kStepQ = 4096, kStep = kStepQ + 512;
constexpr int kBuffers = 3;  // of input rows

// Input rows in shared memory are 16-bit operands, with a pad that keeps the fragments' reads
// free of bank conflicts.  A buffer is the rows, then for every group of columns -8 sum(x) of
// each row, then (8-bit rows) the scales of each 128 columns and row.
__host__ __device__ constexpr int x_pitch(int steps) { return 512 * steps + 64; }
__host__ __device__ constexpr int x_bytes(bool x8, int tile, int rows, int steps, int group) {
  return (rows * x_pitch(steps) + tile * 4 * steps * (256 / group + (x8 ? 2 : 0)) + 127) /
         128 * 128;
}
// Steps that a buffer has room for (16 at most: a warp copies the scales of a chunk at once).
__host__ __device__ constexpr int x_steps_of(int bytes, bool x8, int tile, int rows, int group) {
  const int n = (bytes - 64 * rows) / (512 * rows + tile * 4 * (256 / group + (x8 ? 2 : 0)));
  return n < 16 ? n : 16;
}
// Bytes of the partial sums: of the warps of units cut into `split`, or of a run of pairs that
// the blocks of a cluster hand over at once.
constexpr int kHandOver = 8;
__host__ __device__ constexpr int sum_bytes(int nt, int split, int cluster) {
  const int pairs = kWarps - kWarps / split;
  return (cluster > 1 && pairs < kHandOver ? kHandOver : pairs) * 8 * nt * 32 * 4;
}

// What `rest` < n items take on n blocks (or clusters) when each is cut into 2^cut units, in half
// steps: the rounds of units times the unit's steps and half a step beside them.  Where a chunk of
// input rows (x_steps) is less than kDepth steps for a share, every step waits for its rows, and
// counts one and a half.
__host__ __device__ __forceinline__ int cost_of(int rest, int n, int steps, int x_steps, int cut) {
  const int mine = (steps + (1 << cut) - 1) >> cut, chunk = x_steps >> cut;
  return ((rest << cut) + n - 1) / n * (mine * (chunk < kDepth && chunk < mine ? 3 : 2) + 1);
}

// Asynchronous copies to shared memory.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
// Eight columns of an input row on their way into a slot of 16 bytes (8-bit rows, which start on
// 8 bytes, into its upper half).
template <bool kX8>
__device__ __forceinline__ void copy_x(uint32_t slot, const void* src) {
  if constexpr (kX8)
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(slot + 8), "l"(src) : "memory");
  else
    copy16(slot, src);
}
// The slot's eight columns as operands: bf16 times 2^65, or fp16; returns the sum of the columns
// themselves (each is scaled back before it is added: 128 operands of one sign may add up to more
// than fp32 holds), infinite or NaN where an operand is.
template <bool kX8>
__device__ __forceinline__ float make_x(uint32_t slot) {
  uint32_t v[4];
  float sum = 0.f;
  if constexpr (kX8) {
    uint32_t lo, hi;
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(lo), "=r"(hi) : "r"(slot + 8) : "memory");
    const uint16_t p[4] = {(uint16_t)lo, (uint16_t)(lo >> 16), (uint16_t)hi, (uint16_t)(hi >> 16)};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(v[i]) : "h"(p[i]));
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&v[i]));
      sum += f.x + f.y;
    }
  } else {
    const __nv_bfloat162 k = __floats2bfloat162_rn(0x1p65f, 0x1p65f);
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                 : "r"(slot)
                 : "memory");
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 r = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&v[i]), k);
      v[i] = *reinterpret_cast<const uint32_t*>(&r);
      sum = fmaf(__uint_as_float(v[i] << 16), 0x1p-65f, sum);
      sum = fmaf(__uint_as_float(v[i] & 0xffff0000u), 0x1p-65f, sum);
    }
  }
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(slot), "r"(v[0]), "r"(v[1]),
               "r"(v[2]), "r"(v[3])
               : "memory");
  return sum;
}
__device__ __forceinline__ void zero_x(uint32_t slot) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(slot), "r"(0) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// All but the newest kLeft groups have arrived.
template <int kLeft>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}

// d = a b + c
template <bool kHalf>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                    uint32_t b1, const float (&c)[4]) {
  if constexpr (kHalf)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]),
          "f"(c[2]), "f"(c[3]));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]),
          "f"(c[2]), "f"(c[3]));
}

// The four A registers of one word of codes, as subnormal numbers: in the fragment's rows g the
// code of row g and 16 times that of row g + 8, in its rows g + 8 the code of row g alone.
__device__ __forceinline__ void widen(uint32_t w, uint32_t (&a)[4]) {
  a[0] = w & 0x00ff00ffu;
  a[1] = w & 0x000f000fu;
  a[2] = __byte_perm(w, 0, 0x4341);
  a[3] = a[2] & 0x000f000fu;
}
// What makes codes of them again, for rows g and rows g + 8.
template <bool kX8>
__device__ __forceinline__ float code_unit(bool upper) {
  const float u = kX8 ? 0x1p24f : 0x1p68f;  // (133 - 65)
  return upper ? u * 0.0625f : u;
}

__device__ __forceinline__ float clip(float v, float c) { return v > c ? c : v < -c ? -c : v; }

// A unit of work of a block.
struct Item {
  int e = 0, tile_rows = 0;
  int pair0 = 0, n_pairs = 0;  // the unit's pairs of blocks of 16 rows
  int log2 = 0, split = 1;     // warps that share the columns of a pair
  int steps = 0;               // of 256 columns, of the longest share
  int x_steps = 0;             // steps (of all shares together) of a chunk of input rows
  bool shared = false;
  int in_row0 = 0, out_row0 = 0;  // (rows are below 2^31: checked on the host)
};

template <int kNt, bool kX8, int kGroup, bool kCluster>
__global__ void __launch_bounds__(kThreads, 1) w4_kernel(const Args a) {
  constexpr int kTile = 8 * kNt;        // rows of a group that one item takes
  constexpr int kSteps = 256 / kGroup;  // groups in a step
  constexpr int kEl = kX8 ? 1 : 2;      // bytes of an input element
  using Count = std::conditional_t<kNt == 1, int, int64_t>;  // tiles; light ones in the upper half
  __shared__ Count s_warp[kWarps];
  __shared__ int32_t s_x_steps[kTile + 1];  // steps of a chunk of so many rows
  extern __shared__ __align__(1024) char s_ring[];  // the rings, the rows' buffers, partial sums
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int n_all = a.n_groups + a.has_shared;
  // the groups' first tiles of more than 8 rows (kNt = 1: all tiles), their first tiles of at most
  // 8, which come behind all others, their first rows, and their rows
  int32_t* const s_first = reinterpret_cast<int32_t*>(s_ring + a.tables);
  int32_t* const s_light = s_first + n_all + 1;
  int32_t* const s_row = s_light + n_all + 1;
  int32_t* const s_rows = s_row + n_all;
  __shared__ uint64_t s_full[kBuffers], s_free[kBuffers];
  __shared__ int s_abort;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kBuffers; ++i) {
      mbar::init(&s_full[i], kWarps);
      mbar::init(&s_free[i], kWarps);
    }
    s_abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  pdl_wait();

  // rows of group e, the first of them in `first`; -1 where its offsets are wrong
  auto group_rows = [&](int e, int& first) -> int {
    first = 0;
    if (e >= a.n_groups) return a.shared_rows;
    if (a.offsets == nullptr) return a.max_rows;
    first = a.offsets[e];
    const int64_t n = (int64_t)a.offsets[e + 1] - first;
    return first < 0 || n < 0 || n > a.max_group_rows || first + n > a.max_rows ? -1 : (int)n;
  };
  // a row index out of range somewhere: each tile looks for it then
  bool bad_index = false;
  if (a.row_index != nullptr) {
    const int n = a.offsets != nullptr ? min(max(a.offsets[a.n_groups], 0), a.max_rows) : a.max_rows;
    if (n > 16 * kThreads) bad_index = true;  // (longer than it is worth: they look anyway)
    for (int i = threadIdx.x; i < n && !bad_index; i += kThreads) {
      const int v = a.row_index[i];
      if (v < 0 || v >= a.x_rows) bad_index = true;
    }
  }
  {
    // tiles of every group, and their exclusive scan
    const int per = (n_all + kThreads - 1) / kThreads;
    const int e0 = threadIdx.x * per;
    Count mine = 0;
    bool bad = false;
    for (int e = e0; e < e0 + per && e < n_all; ++e) {
      int first, n = group_rows(e, first);
      if (n < 0) bad = true, n = 0;
      const int tiles = (n + kTile - 1) / kTile;
      const bool light = kNt > 1 && n % kTile != 0 && n % kTile <= 8;
      s_first[e] = tiles - light;
      s_light[e] = light;
      s_row[e] = first;
      s_rows[e] = n;
      mine += tiles - light;
      if constexpr (kNt > 1) mine += (int64_t)light << 32;
    }
    if (bad && blockIdx.x == 0) report_status(a.status, kStatusInvalidInput);
    // (where offsets contradict each other, the last one does not bound the rows looked at above)
    bad_index |= bad;
    if (threadIdx.x >= 1 && threadIdx.x <= kTile)
      s_x_steps[threadIdx.x] = x_steps_of(a.buf_bytes, kX8, kTile, threadIdx.x, kGroup);
    Count incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const Count v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) s_warp[warp] = incl;
    __syncthreads();
    Count sum = incl - mine;
    for (int w = 0; w < warp; ++w) sum += s_warp[w];
    int at = (int)sum, at_light = kNt > 1 ? (int)((int64_t)sum >> 32) : 0;
    for (int e = e0; e < e0 + per && e < n_all; ++e) {
      const int tiles = s_first[e], light = s_light[e];
      s_first[e] = at;
      s_light[e] = at_light;
      at += tiles;
      at_light += light;
    }
    if (threadIdx.x == kThreads - 1) {
      s_first[n_all] = at;
      s_light[n_all] = at_light;
    }
    bad_index = __syncthreads_or(bad_index);
  }
  // The blocks of a cluster work on the same items, each on its run of the steps, k0 onwards.
  const int per = kCluster ? a.cluster : 1, all_steps = (a.ku + 3) / 4, rank = blockIdx.x % per;
  const int k0 = all_steps * rank / per;
  const int n_steps = all_steps * (rank + 1) / per - k0;
  // an item: a tile and a pair of blocks for each warp; those after the last whole round of the
  // blocks are cut into 2^cut units
  const int chunks = (a.pairs + kWarps - 1) / kWarps;
  const int n_blocks = (int)gridDim.x / per, block = (int)blockIdx.x / per;
  const int n_full = s_first[n_all], items = (n_full + s_light[n_all]) * chunks;  // (units are below 2^31: checked on the host)
  const int rest = items % n_blocks, whole = items - rest;
  int cut = 0;
  for (int c = 1; 1 << c <= a.max_split; ++c) {
    const int most = (all_steps + per - 1) / per;  // (the cut is all blocks' alike)
    if (cost_of(rest, n_blocks, most, a.x_steps, c) < cost_of(rest, n_blocks, most, a.x_steps, cut))
      cut = c;
  }
  const int units = whole + (rest << cut);

  // A block's units, one in each round: its place there and back, so that what the costlier tiles
  // at the front take longer is made up for by cheaper ones.  `step` is from one to the next.
  const int first_step = 2 * (n_blocks - block) - 1;
  auto next_unit = [&](int& unit, int& step) {
    unit += step;
    step = 2 * n_blocks - step;
  };
  auto item_at = [&](int unit) {
    Item r;
    int it = unit, part = 0;
    if (unit >= whole) {
      it = whole + ((unit - whole) >> cut);
      part = (unit - whole) & ((1 << cut) - 1);
      r.log2 = cut;
      r.split = 1 << cut;
    }
    int tile = (int)((unsigned)it / (unsigned)chunks);
    r.pair0 = (it - tile * chunks) * kWarps + part * (kWarps >> r.log2);
    r.n_pairs = min(kWarps >> r.log2, a.pairs - r.pair0);
    r.steps = (n_steps + r.split - 1) >> r.log2;
    const bool light = kNt > 1 && tile >= n_full;
    const int32_t* const table = light ? s_light : s_first;
    if (light) tile -= n_full;
    int hi = n_all;  // the group that owns the tile: table[e] <= tile < table[e + 1]
    while (hi - r.e > 1) {
      const int mid = (r.e + hi) >> 1;
      if (table[mid] <= tile)
        r.e = mid;
      else
        hi = mid;
    }
    r.shared = r.e >= a.n_groups;
    const int first = s_row[r.e];
    const int row0 = light ? s_rows[r.e] / kTile * kTile : (tile - table[r.e]) * kTile;
    r.tile_rows = min(kTile, s_rows[r.e] - row0);
    r.x_steps = min(s_x_steps[r.tile_rows], n_steps + r.split - 1) >> r.log2 << r.log2;
    r.out_row0 = (r.shared ? a.shared_out_row0 : first) + row0;
    r.in_row0 = (r.shared ? a.shared_x_row0 : first) + row0;
    return r;
  };
  // the input row of a tile's row r; -1 where its index is out of range
  auto row_of = [&](const Item& im, int r) -> int {
    int v = im.in_row0 + r;
    if (!im.shared && a.row_index != nullptr) v = a.row_index[v];
    return v < 0 || v >= a.x_rows ? -1 : v;
  };

  // ---- input rows, in chunks ----
  // A warp's part of a chunk, of slots of 8 columns: with the rows rounded up to a power of two,
  // `over`, it is row warp % over, and of its runs of 32 slots every (kWarps / over)-th from
  // warp / over.
  char* const s_x = s_ring + kWarps * kDepth * kStep;
  const uint32_t x0 = (uint32_t)__cvta_generic_to_shared(s_x);
  // where a buffer's sums [group][kTile] and scales [128 columns][kTile] begin
  auto sums_of = [](int rows, int x_steps) { return rows * x_pitch(x_steps); };
  auto scales_of = [](int rows, int x_steps) {
    return rows * x_pitch(x_steps) + x_steps * kSteps * kTile * 4;
  };
  int c_it = block, c_go = first_step;  // unit and first step of the chunk to copy next
  int c_s = 0, c_steps = 0, c_log2 = 0, c_rows = 0, c_over = 1, c_x_steps = 0, c_buf = 0;
  uint32_t c_phase = 0;    // of the buffer's last freeing
  const char* c_x = nullptr;  // the warp's row at the next chunk's first column
  const float* c_xs = nullptr;
  int n_copied = 0;        // chunks
  // of the two chunks copied last: rows, slots of a row, and those before the last column
  int d_rows[2] = {0, 0}, d_over[2] = {1, 1}, d_steps[2] = {0, 0};
  int d_slots[2] = {0, 0}, d_inside[2] = {0, 0};
  bool dead = false;  // a wait ran out
  auto copy_chunk = [&]() {
    if (c_it >= units) return;
    if (c_s == 0) {
      const Item im = item_at(c_it);
      c_steps = im.steps;
      c_log2 = im.log2;
      c_rows = im.tile_rows;
      c_x_steps = im.x_steps;
      c_over = 1 << (32 - __clz(c_rows - 1));
      const int r = min(warp & (c_over - 1), c_rows - 1);
      const int64_t row = max(row_of(im, r), 0);
      c_x = static_cast<const char*>(a.x) + (row * a.cols + 256 * k0 + 8 * lane) * kEl;
      c_xs = kX8 ? a.x_scale + row * a.xs_ld + (2 * k0 + lane) * a.xs_step : nullptr;
    }
    const int st0 = c_s << c_log2, pitch = x_pitch(c_x_steps);
    const int slots = min(c_x_steps, n_steps - st0) * 32;
    const int inside = min(slots, (a.cols - 256 * (k0 + st0)) >> 3);
    // every warp is done with what the buffer held
    if (n_copied >= kBuffers && !dead)
      dead = !__all_sync(0xffffffffu, mbar::wait(&s_free[c_buf], c_phase, &s_abort, a.status));
    const int r = warp & (c_over - 1);
    if (r < c_rows) {
      const uint32_t to = x0 + c_buf * a.buf_bytes, at = to + r * pitch + 16 * lane;
      const int first = warp / c_over * 32, turn = kWarps / c_over * 32;
      for (int i = first; i + lane < inside; i += turn) copy_x<kX8>(at + 16 * i, c_x + 8 * kEl * i);
      if (kX8 && first == 0 && 16 * lane < inside)
        copy4(to + scales_of(c_rows, c_x_steps) + (lane * kTile + r) * 4, c_xs);
    }
    c_x += c_x_steps * 256 * kEl;
    if (kX8) c_xs += 2 * c_x_steps * a.xs_step;
    d_rows[1] = d_rows[0], d_over[1] = d_over[0], d_steps[1] = d_steps[0];
    d_slots[1] = d_slots[0], d_inside[1] = d_inside[0];
    d_rows[0] = c_rows, d_over[0] = c_over, d_steps[0] = c_x_steps;
    d_slots[0] = slots, d_inside[0] = inside;
    if (++c_buf == kBuffers) {
      c_buf = 0;
      if (n_copied >= kBuffers) c_phase ^= 1;
    }
    copies_commit();  // a group of its own: whichever steps follow, the waits for theirs cover it
    ++n_copied;
    c_s += c_x_steps >> c_log2;
    if (c_s >= c_steps) {
      c_s = 0;
      next_unit(c_it, c_go);
    }
  };
  // Operands, and sums by groups, of the warp's part of a chunk that has landed: the chunk
  // copied last, or the one before it.
  int m_buf = 0, n_made = 0;
  auto make_chunk = [&]() {
    if (n_made >= n_copied) return;
    const bool older = n_copied - n_made == 2;
    const int rows = older ? d_rows[1] : d_rows[0], slots = older ? d_slots[1] : d_slots[0];
    const int inside = older ? d_inside[1] : d_inside[0], over = older ? d_over[1] : d_over[0];
    const int x_steps = older ? d_steps[1] : d_steps[0], pitch = x_pitch(x_steps);
    const uint32_t at = x0 + m_buf * a.buf_bytes, sums = at + sums_of(rows, x_steps);
    constexpr int kLanes = kGroup / 8;  // slots of a group
    const int r = warp & (over - 1);
    if (r < rows) {
      for (int i = warp / over * 32 + lane; i - lane < slots; i += kWarps / over * 32) {
        float sum = 0.f;
        if (i < inside)
          sum = make_x<kX8>(at + r * pitch + 16 * i);
        else if (i < slots)
          zero_x(at + r * pitch + 16 * i);
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (i % kLanes == 0 && i < slots)
          asm volatile("st.shared.f32 [%0], %1;" ::"r"(sums + (i / kLanes * kTile + r) * 4),
                       "f"(sum * (-8.f / code_unit<kX8>(false)))
                       : "memory");
      }
    }
    __syncwarp();
    if (lane == 0) mbar::arrive(&s_full[m_buf]);
    m_buf = m_buf + 1 == kBuffers ? 0 : m_buf + 1;
    ++n_made;
  };

  // ---- weights: the warp's ring; step f_s of the share of unit f_it is fetched next ----
  char* const s_mine = s_ring + warp * (kDepth * kStep);
  const uint32_t ring0 = (uint32_t)__cvta_generic_to_shared(s_mine) + lane * 16;
  int f_it = block, f_go = first_step;
  int f_plain = 0;                       // steps of the share before its last one
  int f_s = 0, f_steps = 0, f_n = 0;     // then: the step, the unit's steps, and the share's
  int f_last = 0, f_dq = 0, f_ds = 0;    // the last step's place; bytes from a step to the next
  const char *fq0 = nullptr, *fq1 = nullptr, *fs = nullptr;
  const int s_m = lane >= 2 * kSteps, s_c = lane % (2 * kSteps);  // the lane's 16 bytes of scales
  // the warp's share and pair of a unit
  auto steps_of = [&](const Item& im) {
    const int ks = warp & (im.split - 1);
    return warp >> im.log2 < im.n_pairs ? (n_steps - ks + im.split - 1) >> im.log2 : 0;
  };
  auto fetch_item = [&]() {
    f_plain = f_s = f_n = 0;
    f_steps = 1;
    if (f_it >= units) return;
    const Item im = item_at(f_it);
    const int ks = warp & (im.split - 1), pair = im.pair0 + (warp >> im.log2);
    f_steps = im.steps;
    f_n = steps_of(im);
    f_plain = f_s = max(f_n - 1, 0);
    f_last = k0 + f_s * im.split + ks;
    f_dq = 2048 * im.split;
    f_ds = 32 * kSteps * im.split;
    const int64_t blk = (int64_t)im.e * a.parts * a.rb;
    const int64_t b0 = blk + (a.parts == 2 ? pair : 2 * pair);
    const int64_t b1 = blk + (a.parts == 2 ? a.rb + pair : min(2 * pair + 1, a.rb - 1));
    fq0 = reinterpret_cast<const char*>(a.q + (b0 * a.ku + 4 * (k0 + ks)) * 32 + lane);
    fq1 = reinterpret_cast<const char*>(a.q + (b1 * a.ku + 4 * (k0 + ks)) * 32 + lane);
    fs = reinterpret_cast<const char*>(a.scale + ((s_m ? b1 : b0) * a.ng + (k0 + ks) * kSteps) * 8 + 4 * s_c);
  };
  // the next step into the ring at `at` (an empty group where there is none)
  auto fetch = [&](int at) {
    const uint32_t dst = ring0 + at;
    if (f_plain > 0) {
      --f_plain;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        copy16(dst + 512 * u, fq0 + 512 * u);
        copy16(dst + 2048 + 512 * u, fq1 + 512 * u);
      }
      if (lane < 4 * kSteps) copy16(dst + kStepQ, fs);
      fq0 += f_dq;
      fq1 += f_dq;
      fs += f_ds;
    } else {
      if (f_s < f_n) {
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          if (4 * f_last + u >= a.ku) break;  // (old codes meet zero columns there)
          copy16(dst + 512 * u, fq0 + 512 * u);
          copy16(dst + 2048 + 512 * u, fq1 + 512 * u);
        }
        if (lane < 4 * kSteps && f_last * kSteps + s_c / 2 < a.ng) copy16(dst + kStepQ, fs);
      }
      if (++f_s >= f_steps) {
        next_unit(f_it, f_go);
        fetch_item();
      }
    }
    copies_commit();
  };

  if ((int)blockIdx.x * kWarps + warp == a.give_up) {
    dead = true;
    *(volatile int*)&s_abort = 1;
    __threadfence_block();
    report_status(a.status, kStatusTimeout);
  }
  fetch_item();
  copy_chunk();
  fetch(0);
  copy_chunk();
#pragma unroll
  for (int p = 1; p < kDepth; ++p) fetch(p * kStep);
  copies_wait<kDepth - 1>();  // the first chunk
  make_chunk();
  int buf = 0, at = 0;
  uint32_t x_phase = 0;
  for (int unit = block, go = first_step; unit < units; next_unit(unit, go)) {
    const Item im = item_at(unit);
    const int ks = warp & (im.split - 1), pair = im.pair0 + (warp >> im.log2);
    const int n_mine = steps_of(im), chunk = im.x_steps >> im.log2;
    float acc[2][kNt][4];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int n = 0; n < kNt; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[m][n][i] = 0.f;
    // the item's steps with kN blocks of 8 rows
    auto steps = [&](auto blocks) {
      constexpr int kN = decltype(blocks)::value;
      // What a column of an mma holds depends on its own row alone: rows behind the tile's last
      // one read that one again, and their sums are not stored.
      int x_off[kN];
#pragma unroll
      for (int n = 0; n < kN; ++n)
        x_off[n] = min(8 * n + g, im.tile_rows - 1) * x_pitch(im.x_steps) + 16 * t;
      for (int c0 = 0; c0 < im.steps; c0 += chunk) {
        if (!dead)
          dead = !__all_sync(0xffffffffu, mbar::wait(&s_full[buf], x_phase, &s_abort, a.status));
        const int n_now = dead ? 0 : n_mine, end = min(c0 + chunk, im.steps);
        const char* px = s_x + buf * a.buf_bytes + ks * 512;
        const char* po = s_x + buf * a.buf_bytes + sums_of(im.tile_rows, im.x_steps) +
                         (ks * kSteps * kTile + 2 * t) * 4;
        const char* pxs = s_x + buf * a.buf_bytes + scales_of(im.tile_rows, im.x_steps) +
                          (2 * ks * kTile + 2 * t) * 4;
        // a first step, to let the other warps end the chunk before; then the next chunk but one
        // is copied (and where a chunk is short, the next one made), and the other steps follow
        int s = c0;
        bool copied = false;
        for (int stop = c0 + 1;; stop = end) {
          for (; s < stop; ++s) {
            copies_wait<kDepth - 1>();
            __syncwarp();  // other lanes' scales
            if (s < n_now) {
              const char* pq = s_mine + at + lane * 16;
              const uint32_t* ps = reinterpret_cast<const uint32_t*>(s_mine + at + kStepQ) + g;
              // of the step's groups, the last there is
              const int st = k0 + (s << im.log2) + ks, g_last = a.ng - 1 - st * kSteps;
              float part[2][kN][4];
              uint4 w[2];
#pragma unroll
              for (int h = 0; h < 8; ++h) {  // 32 columns each
                if (h == 4 && 256 * st + 128 >= a.cols) break;
                if (h % 2 == 0) {
                  w[0] = *reinterpret_cast<const uint4*>(pq + 256 * h);
                  w[1] = *reinterpret_cast<const uint4*>(pq + 256 * h + 2048);
                }
                uint4 b[kN];
#pragma unroll
                for (int n = 0; n < kN; ++n)
                  b[n] = *reinterpret_cast<const uint4*>(px + x_off[n] + 64 * h);
                float off[kN][4];  // what a group's sums start from
                if (h % (kGroup / 32) == 0) {
#pragma unroll
                  for (int n = 0; n < kN; ++n) {
                    const float2 o = *reinterpret_cast<const float2*>(
                        po + (h / (kGroup / 32) * kTile + 8 * n) * 4);
                    off[n][0] = 17.f * o.x;
                    off[n][1] = 17.f * o.y;
                    off[n][2] = o.x;
                    off[n][3] = o.y;
                  }
                }
#pragma unroll
                for (int j = 0; j < 2; ++j) {
#pragma unroll
                  for (int m = 0; m < 2; ++m) {
                    const uint32_t word = (h & 1) ? (j ? w[m].w : w[m].z) : (j ? w[m].y : w[m].x);
                    uint32_t fa[4];
                    widen(word, fa);
#pragma unroll
                    for (int n = 0; n < kN; ++n)
                      mma<kX8>(part[m][n], fa, j ? b[n].z : b[n].x, j ? b[n].w : b[n].y,
                               j == 0 && h % (kGroup / 32) == 0 ? off[n] : part[m][n]);
                  }
                }
                if ((h + 1) % (kGroup / 32) != 0) continue;
                const int gi = kGroup == 128 ? h / 4 : min(h / (kGroup / 32), g_last);
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                  const uint32_t sw = ps[(m * kSteps + gi) * 8];
                  const float lo = __uint_as_float(sw << 16), up = __uint_as_float(sw & 0xffff0000u);
#pragma unroll
                  for (int n = 0; n < kN; ++n) {
                    // rows g, then rows g + 8 (16 times as large)
                    const float s0 = part[m][n][2], s1 = part[m][n][3];
                    const float s2 = part[m][n][0] - s0, s3 = part[m][n][1] - s1;
                    if (kX8) {
                      const float2 xs = *reinterpret_cast<const float2*>(pxs + (h / 4 * kTile + 8 * n) * 4);
                      acc[m][n][0] = fmaf(s0, lo * xs.x, acc[m][n][0]);
                      acc[m][n][1] = fmaf(s1, lo * xs.y, acc[m][n][1]);
                      acc[m][n][2] = fmaf(s2, up * xs.x, acc[m][n][2]);
                      acc[m][n][3] = fmaf(s3, up * xs.y, acc[m][n][3]);
                    } else {
                      acc[m][n][0] = fmaf(s0, lo, acc[m][n][0]);
                      acc[m][n][1] = fmaf(s1, lo, acc[m][n][1]);
                      acc[m][n][2] = fmaf(s2, up, acc[m][n][2]);
                      acc[m][n][3] = fmaf(s3, up, acc[m][n][3]);
                    }
                  }
                }
              }
            }
            px += 512 << im.log2;
            po += kSteps * kTile * 4 << im.log2;
            if (kX8) pxs += 2 * kTile * 4 << im.log2;
            __syncwarp();  // the slot's scales have been read
            fetch(at);
            at = at + kStep == kDepth * kStep ? 0 : at + kStep;
          }
          if (copied) break;
          copied = true;
          if (end - c0 < kDepth) {
            copies_wait<0>();
            make_chunk();
          }
          copy_chunk();
        }
        if (end - c0 >= kDepth) make_chunk();  // the next chunk landed a chunk ago
        if (lane == 0) mbar::arrive(&s_free[buf]);
        if (++buf == kBuffers) {
          buf = 0;
          x_phase ^= 1;
        }
      }
    };
    const int n_act = (im.tile_rows + 7) / 8;
    if constexpr (kNt == 1) {
      steps(std::integral_constant<int, 1>{});
    } else {
      if (n_act == 1)
        steps(std::integral_constant<int, 1>{});
      else
        steps(std::integral_constant<int, 2>{});
    }
    // Where a wait of any of the block's warps has run out, rows may be missing or may have been
    // overwritten under another warp: all that the block still stores or hands over is NaN, so that
    // a caller without a status word learns of it too.
    dead = __any_sync(0xffffffffu, dead || *(volatile int*)&s_abort != 0);
    if (dead) {
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int n = 0; n < kNt; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[m][n][i] = NAN;
    }
    if (im.split > 1) {
      __syncthreads();  // the last unit's sums have been read
      // the warps but the first of each pair leave theirs
      const int place = (warp >> im.log2) * (im.split - 1) + ks - 1;
      float* sums = reinterpret_cast<float*>(s_x + kBuffers * a.buf_bytes) +
                    place * (8 * kNt * 32) + lane;
      if (ks != 0) {
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int n = 0; n < kNt; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) sums[((m * kNt + n) * 4 + i) * 32] = acc[m][n][i];
      }
      __syncthreads();
      if (ks == 0) {
        for (int o = 1; o < im.split; ++o) {
          const float* other = sums + o * (8 * kNt * 32);
#pragma unroll
          for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int n = 0; n < kNt; ++n)
#pragma unroll
              for (int i = 0; i < 4; ++i) acc[m][n][i] += other[((m * kNt + n) * 4 + i) * 32];
        }
      }
    }
    if constexpr (kCluster) {
      // the first block of the cluster adds the others' sums, in order, some pairs at a time
      cg::cluster_group cluster = cg::this_cluster();
      const int mine = warp >> im.log2;
      float* sums = reinterpret_cast<float*>(s_x + kBuffers * a.buf_bytes) +
                    mine % kHandOver * (8 * kNt * 32) + lane;
      if (im.split > 1) __syncthreads();  // the block's own sums have been read
      for (int first = 0; first < kWarps >> im.log2; first += kHandOver) {
        const bool now = ks == 0 && mine / kHandOver * kHandOver == first;
        if (now && rank != 0) {
#pragma unroll
          for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int n = 0; n < kNt; ++n)
#pragma unroll
              for (int i = 0; i < 4; ++i) sums[((m * kNt + n) * 4 + i) * 32] = acc[m][n][i];
        }
        cluster.sync();
        if (now && rank == 0) {
          for (int o = 1; o < per; ++o) {
            const float* other = cluster.map_shared_rank(sums, o);
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
              for (int n = 0; n < kNt; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[m][n][i] += other[((m * kNt + n) * 4 + i) * 32];
          }
        }
        cluster.sync();
      }
      if (rank != 0) continue;
    }
    if (n_mine == 0 || ks != 0) continue;
    // rows 16 b + g and + 8 of block b, and (without SwiGLU) of the block behind it
    const int row0 = 16 * (a.parts == 2 ? pair : 2 * pair) + g;
#pragma unroll
    for (int n = 0; n < kNt; ++n) {
      if (8 * n >= im.tile_rows) break;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int r = 8 * n + 2 * t + j;
        if (r >= im.tile_rows) continue;
        float v[2][2];  // [block][row]
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          v[m][0] = acc[m][n][j] * code_unit<kX8>(false);
          v[m][1] = acc[m][n][2 + j] * code_unit<kX8>(true);
        }
        if (a.parts == 2) {
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            float gate = v[0][q], up = v[1][q];
            if (a.clamp > 0.f) {
              gate = clip(gate, a.clamp);
              up = clip(up, a.clamp);
            }
            v[0][q] = gate / (1.f + expf(-gate)) * up;
          }
        } else if (a.relu) {
#pragma unroll
          for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int q = 0; q < 2; ++q) v[m][q] = v[m][q] < 0.f ? 0.f : v[m][q];
        }
        // a row index out of range is reported, and its row reads as zeros
        if (bad_index && row_of(im, r) < 0) {
          report_status(a.status, kStatusInvalidInput);
          v[0][0] = v[0][1] = v[1][0] = v[1][1] = 0.f;
        }
        const int64_t o = (int64_t)(im.out_row0 + r) * a.rows + row0;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          if (a.parts == 2 && q >= 2) break;
          if (row0 + 8 * q >= a.rows) break;
          if (a.out_f32)
            static_cast<float*>(a.out)[o + 8 * q] = v[q >> 1][q & 1];
          else
            static_cast<__nv_bfloat16*>(a.out)[o + 8 * q] = __float2bfloat16_rn(v[q >> 1][q & 1]);
        }
      }
    }
  }
  copies_wait<0>();  // nothing is in flight when the block ends
}

template <int kNt, bool kX8, int kGroup, bool kCluster>
cudaError_t launch_one(const Args& a, int grid, size_t smem, cudaStream_t stream) {
  const auto kernel = w4_kernel<kNt, kX8, kGroup, kCluster>;
  static std::atomic<bool> ready[64];  // the attribute is set once on each device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !ready[dev].load(std::memory_order_relaxed)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kDynamicSmem);
    if (e != cudaSuccess) return e;
    if (dev < 64) ready[dev].store(true, std::memory_order_relaxed);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = 32 * kWarps;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = a.cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = kCluster ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

template <int kNt, bool kX8, bool kCluster>
cudaError_t launch_group(const Args& a, int group, int grid, size_t smem, cudaStream_t stream) {
  return group == 32   ? launch_one<kNt, kX8, 32, kCluster>(a, grid, smem, stream)
         : group == 64 ? launch_one<kNt, kX8, 64, kCluster>(a, grid, smem, stream)
                       : launch_one<kNt, kX8, 128, kCluster>(a, grid, smem, stream);
}

template <bool kX8>
cudaError_t launch_tile(const Args& a, int nt, int group, int grid, size_t smem,
                        cudaStream_t stream) {
  if (nt == 1)
    return a.cluster > 1 ? launch_group<1, kX8, true>(a, group, grid, smem, stream)
                         : launch_group<1, kX8, false>(a, group, grid, smem, stream);
  return a.cluster > 1 ? launch_group<2, kX8, true>(a, group, grid, smem, stream)
                       : launch_group<2, kX8, false>(a, group, grid, smem, stream);
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
  a.x_rows = (int)p.x_rows;
  a.row_index = p.row_index;
  a.offsets = p.offsets;
  a.n_groups = p.n_groups;
  a.has_shared = p.has_shared;
  a.max_rows = (int)p.max_rows;
  a.max_group_rows = (int)p.max_group_rows;
  a.shared_rows = (int)p.shared_rows;
  a.shared_x_row0 = (int)p.shared_x_row0;
  a.shared_out_row0 = (int)p.shared_out_row0;
  a.pairs = p.parts == 2 ? a.rb : (a.rb + 1) / 2;
  a.relu = p.relu;
  a.clamp = p.clamp;
  a.out = p.out;
  a.out_f32 = p.out_f32;
  a.status = p.status;
  a.give_up = p.give_up;
  // rows of a tile: enough for the largest group there can be, 16 at most
  const int64_t most = p.has_shared ? (p.shared_rows > p.max_group_rows ? p.shared_rows : p.max_group_rows)
                                    : p.max_group_rows;
  const int nt = most <= 8 ? 1 : 2;
  const bool x8 = p.x_scale != nullptr;
  const int sms = tc::num_sms();
  const int tile = 8 * nt, n_steps = (a.ku + 3) / 4;
  const int rows = (int)(most < tile ? most : tile);  // the most of a tile
  // shared memory: the rings, the partial sums, and three buffers of input rows, in which a
  // chunk of a step for each share of a cut item has to fit
  const int table_bytes = 4 * (4 * (p.n_groups + p.has_shared) + 2);
  const auto buffer = [&](int split, int cluster) {
    const int room = (kDynamicSmem - table_bytes - kWarps * kDepth * kStep -
                      sum_bytes(nt, split, cluster)) / kBuffers / 128 * 128;
    const int all = x_bytes(x8, tile, rows, n_steps < 16 ? n_steps : 16, p.group);
    return room < all ? room : all;
  };
  // Clusters of 1 to 8 blocks, and the finest cut that there is room for, whichever has the items
  // that are expected done first; a unit's hand-over takes about a step.  Clusters lie within the
  // device's eight groups of SMs: of 148 SMs, 18 in each are counted on (all, for 1, 2 or 4).
  const int64_t shared_tiles = p.has_shared ? (p.shared_rows + tile - 1) / tile : 0;
  const int64_t reached = p.max_rows < p.n_groups ? p.max_rows : p.n_groups;
  const int64_t chunks = (a.pairs + kWarps - 1) / kWarps;
  const int64_t expected = ((p.offsets == nullptr ? (p.max_rows + tile - 1) / tile : reached) +
                            shared_tiles) * chunks;
  const auto clusters_of = [&](int c) { return c <= 2 || c == 4 ? sms / c : sms / 8 / c * 8; };
  int64_t least = -1;
  for (int c = 1; c <= 8 && c <= n_steps && (c == 1 || c <= sms / 8); ++c) {
    const int n = clusters_of(c), steps = (n_steps + c - 1) / c;
    int rest = INT32_MAX;
    for (int k = 0; 1 << k <= kWarps && 1 << k <= steps; ++k) {
      const int x_steps = x_steps_of(buffer(1 << k, c), x8, tile, rows, p.group);
      if (x_steps < 1 << k) break;
      for (int cut = 0; cut <= k; ++cut)
        rest = std::min(rest, cost_of((int)(expected % n), n, steps, x_steps, cut));
      const int64_t cost = expected / n * cost_of(1, 1, steps, x_steps, 0) + rest +
                           (c > 1 ? (expected + n - 1) / n * 2 : 0);
      if (least < 0 || cost < least) {
        least = cost;
        a.cluster = c;
        a.max_split = 1 << k;
        a.x_steps = x_steps;
      }
    }
  }
  a.buf_bytes = buffer(a.max_split, a.cluster);
  const int64_t tiles = p.max_rows / tile + reached + shared_tiles;
  const int64_t units = tiles * chunks * a.max_split;
  if (units > INT32_MAX) return cudaErrorInvalidValue;
  const int64_t n = clusters_of(a.cluster);
  const int grid = (int)(units < 1 ? 1 : units < n ? units : n) * a.cluster;
  a.tables = kWarps * kDepth * kStep + sum_bytes(nt, a.max_split, a.cluster) +
             kBuffers * a.buf_bytes;
  const size_t bytes = (size_t)a.tables + table_bytes;
  ++*launches;
  return x8 ? launch_tile<true>(a, nt, p.group, grid, bytes, stream)
            : launch_tile<false>(a, nt, p.group, grid, bytes, stream);
}

}  // namespace moe
