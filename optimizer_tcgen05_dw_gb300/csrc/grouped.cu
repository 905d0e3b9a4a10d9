// Linears grouped by expert over ragged token groups: the forward product
// Y_t = W_e X_t and the input gradient dX_t = W_e^T dY_t, t in group e.
//
// One persistent tensor-core kernel on CTA pairs, as the linear step's
// (tc_kernel.cuh: the same ring of TMA stages, two accumulators in tensor
// memory, and roles per warp), with the operands the other way round: the
// WEIGHTS are the 256 rows of the matrix instruction (M) and the TOKENS its
// columns (N).  An expert's tokens then cost what they are, rounded up to 32
// columns, where token rows would be rounded up to 256; a group is cut into
// equal column tiles of at most 256 (N of each instruction is chosen per
// tile), so neither short groups nor ragged ends multiply padding.
//   forward  A = W_e rows [128 n x 64 k] per CTA, K-major;
//            B = X rows [up to 128 t x 64 k] per CTA, K-major.
//   dX       A = W_e^T [128 k x 64 n] per CTA, MN-major (read as stored);
//            B = dY rows [up to 128 t x 64 n] per CTA, K-major.
// B rows past a group's end hold other groups' tokens: their columns of the
// accumulator are not stored, and columns do not mix.  The reduction's ragged
// end is zero in both operands (out-of-range reads of the tensor maps; in dX
// the weights' map has the experts as a dimension of its own, so rows past N
// are zeros and not the next expert's).
//
// The group offsets are read on the device (no host synchronisation, so calls
// can be captured in a graph): every CTA builds the same table of column tiles
// from them.  Offsets that leave [0, T] are clamped to it, those that decrease
// count as the largest before them, and either is reported in the status word.
// Rows that belong to no group are set to zero.
#include <cuda_bf16.h>

#include "launch.h"
#include "tc_kernel.cuh"

namespace forge {

namespace {

constexpr int kGStages = 6;
constexpr int kGA = kTileM * kBlockK * 2;        // bytes of A per stage and CTA (128 rows)
constexpr int kGB = (kTileN / 2) * kBlockK * 2;  // of B, at most (128 tokens)
constexpr int kGThreads = 32 * (2 + kNumEpiWarps);
struct GroupTable {
  int32_t off[kMaxGroups + 1];   // first token row of each group
  int32_t tile[kMaxGroups + 1];  // first column tile of each group
  int32_t bad;                   // an offset was out of order or range
};
constexpr int kGSmem = kGStages * (kGA + kGB) + 512 + static_cast<int>(sizeof(GroupTable)) + 1024;
static_assert(kGSmem <= 232448, "dynamic shared memory limit");

// One unit of work: 256 features from f0 of `cols` tokens from t0 of expert e.
struct GroupUnit {
  int e, f0, t0, cols, tend;
};

__device__ __forceinline__ GroupUnit group_unit(int u, const GroupedParams& p, const GroupTable& g) {
  GroupUnit r;
  const int x = u / p.tiles_f;  // column tiles before it, had every group whole rows of units
  int lo = 0, hi = p.groups - 1;
  while (lo < hi) {  // the last group whose first tile is not past x (the empty ones share theirs with it)
    const int mid = (lo + hi + 1) >> 1;
    if (g.tile[mid] <= x) lo = mid;
    else hi = mid - 1;
  }
  r.e = lo;
  const int nt = g.tile[lo + 1] - g.tile[lo];
  int tt, tf;
  tile_coords_of(u - g.tile[lo] * p.tiles_f, nt, p.tiles_f, tt, tf);
  const int cnt = g.off[lo + 1] - g.off[lo];
  const int w = ((cnt + nt - 1) / nt + 31) & ~31;  // <= 256, and (nt - 1) w < cnt
  r.f0 = tf * kPairM;
  r.t0 = g.off[lo] + tt * w;
  r.tend = min(r.t0 + w, g.off[lo + 1]);
  r.cols = (r.tend - r.t0 + 31) & ~31;
  return r;
}

// The table of the groups, by the whole CTA.
__device__ __forceinline__ void build_groups(const GroupedParams& p, GroupTable& g) {
  if (threadIdx.x == 0) g.bad = 0;
  __syncthreads();
  for (int i = threadIdx.x; i <= p.groups; i += blockDim.x) {
    const int raw = p.offsets[i], prev = i > 0 ? p.offsets[i - 1] : 0;
    g.off[i] = min(max(raw, 0), p.T);
    if (raw < prev || raw < 0 || raw > p.T) g.bad = 1;
  }
  __syncthreads();
  if (threadIdx.x < 32) {
    if (g.bad && threadIdx.x == 0) {
      for (int i = 1; i <= p.groups; ++i) g.off[i] = max(g.off[i], g.off[i - 1]);
      atomicCAS(p.status, 0u, static_cast<uint32_t>(kStatusInvalid));
    }
    __syncwarp();
    int base = 0;
    for (int i = 0; i < p.groups; i += 32) {
      const int e = i + threadIdx.x;
      const int n = e < p.groups ? (g.off[e + 1] - g.off[e] + kTileN - 1) / kTileN : 0;
      int incl = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xFFFFFFFFu, incl, o);
        if (static_cast<int>(threadIdx.x) >= o) incl += v;
      }
      if (e < p.groups) g.tile[e] = base + incl - n;
      base += __shfl_sync(0xFFFFFFFFu, incl, 31);
    }
    if (threadIdx.x == 0) g.tile[p.groups] = base;
  }
  __syncthreads();
}

// Which of the token maps (boxes of 16, 32, 64, 128 rows) covers half the columns.
__device__ __forceinline__ int box_of(int cols) {
  const int half = cols >> 1;
  return half <= 16 ? 0 : (half <= 32 ? 1 : (half <= 64 ? 2 : 3));
}

template <bool DGRAD>
__device__ void grouped_producer(const CUtensorMap* mW, const CUtensorMap* mT, const GroupedParams& p,
                                 const GroupTable& g, uint8_t* smA, uint8_t* smB, SharedState* ss, uint32_t rank) {
  uint32_t it = 0, issued_mask = 0, last_parity = 0;
  const uint32_t full0 = ptx::mapa(ptx::smem_addr(&ss->full[0]), 0);
  const int units = g.tile[p.groups] * p.tiles_f;
  if (!p.skip_loads) {
    for (int u = pair_id(); u < units; u += num_pairs()) {
      const GroupUnit q = group_unit(u, p, g);
      const int m0 = q.f0 + static_cast<int>(rank) * kTileM;
      const int t0 = q.t0 + static_cast<int>(rank) * (q.cols >> 1);
      const int box = box_of(q.cols);
      const uint32_t bytes = 2u * (kGA + ((16u << box) * kBlockK * 2));
      for (int kb = 0; kb < p.num_kb; ++kb, ++it) {
        const int s = static_cast<int>(it % kGStages);
        const uint32_t ph = (it / kGStages) & 1u;
        if (!bounded_wait(&ss->empty[s], ph ^ 1u, p, ss)) goto drain;
        const uint32_t bar = full0 + static_cast<uint32_t>(s) * 8u;
        if (rank == 0) ptx::mbar_arrive_expect_tx(&ss->full[s], bytes);
        uint8_t* a = smA + s * kGA;
        if (!DGRAD) {
          ptx::tma_load_2d_pair(mW, bar, a, kb * kBlockK, q.e * p.w_rows + m0);
        } else if (p.w3d) {
          ptx::tma_load_4d_pair(mW, bar, a, 0, kb * kBlockK, m0 / 64, q.e);
        } else {
          ptx::tma_load_3d_pair(mW, bar, a, m0, kb * kBlockK, q.e);
          ptx::tma_load_3d_pair(mW, bar, a + 64 * kBlockK * 2, m0 + 64, kb * kBlockK, q.e);
        }
        ptx::tma_load_2d_pair(mT + box, bar, smB + s * kGB, kb * kBlockK, t0);
        issued_mask |= 1u << s;
        last_parity = (last_parity & ~(1u << s)) | (ph << s);
      }
    }
  }
drain:
  if (rank == 0)  // every issued copy lands before the pair can exit
    for (int s = 0; s < kGStages; ++s)
      if (issued_mask & (1u << s)) bounded_wait(&ss->full[s], (last_parity >> s) & 1u, p, ss, false);
}

template <bool DGRAD>
__device__ void grouped_mma(const GroupedParams& p, const GroupTable& g, uint8_t* smA, uint8_t* smB,
                            SharedState* ss) {
  uint32_t it = 0;
  int local = 0;
  const int units = g.tile[p.groups] * p.tiles_f;
  for (int u = pair_id(); u < units; u += num_pairs(), ++local) {
    const int cols = group_unit(u, p, g).cols;
    const int acc = local & 1;
    const uint32_t aph = (static_cast<uint32_t>(local) >> 1) & 1u;
    if (!bounded_wait(&ss->tmem_empty[acc], aph ^ 1u, p, ss)) goto done;
    ptx::tc_fence_after();
    const uint32_t idesc = ptx::idesc_bf16_f32(kPairM, cols, DGRAD, false);
    const uint32_t d_tmem = ss->tmem_base + static_cast<uint32_t>(acc * kTileN);
    for (int kb = 0; kb < p.num_kb; ++kb, ++it) {
      const int s = static_cast<int>(it % kGStages);
      const uint32_t ph = (it / kGStages) & 1u;
      if (!bounded_wait(&ss->full[s], ph, p, ss)) goto done;
      ptx::tc_fence_after();
      const uint32_t a0 = ptx::smem_addr(smA + s * kGA), b0 = ptx::smem_addr(smB + s * kGB);
#pragma unroll
      for (int kk = 0; kk < kBlockK / 16; ++kk) {
        const uint64_t adesc = DGRAD ? ptx::smem_desc_sw128(a0 + kk * 2048, kBlockK * 128, 1024)
                                     : ptx::smem_desc_sw128(a0 + kk * 32, 16, 1024);
        ptx::mma_bf16_pair(d_tmem, adesc, ptx::smem_desc_sw128(b0 + kk * 32, 16, 1024), idesc,
                           (kb | kk) != 0 ? 1u : 0u);
      }
      ptx::mma_commit_pair_multicast(&ss->empty[s], 0x3);
    }
    ptx::mma_commit_pair_multicast(&ss->tmem_full[acc], 0x3);
  }
done:
  ptx::mma_commit_pair_multicast(&ss->mma_done, 0x1);
  bounded_wait(&ss->mma_done, 0u, p, ss, false);
}

// A lane holds one feature of 16 tokens; out is token-major.  Neighbouring
// lanes swap halves of each pair of tokens, so that each stores two features of
// one token: a warp's store covers 64 contiguous bytes of two rows.
__device__ __forceinline__ void grouped_epilogue(const GroupedParams& p, const GroupTable& g, SharedState* ss,
                                                 int warp, int lane, uint32_t rank) {
  const int quarter = warp & 3, half = (warp - 2) >> 2;
  const uint32_t empty0 = ptx::mapa(ptx::smem_addr(&ss->tmem_empty[0]), 0);
  const int units = g.tile[p.groups] * p.tiles_f;
  const int64_t F = p.F;
  const bool odd = lane & 1;
  int local = 0;
  for (int u = pair_id(); u < units; u += num_pairs(), ++local) {
    const GroupUnit q = group_unit(u, p, g);
    const int acc = local & 1;
    const uint32_t aph = (static_cast<uint32_t>(local) >> 1) & 1u;
    bool ok = true;
    if (warp == 2 && lane == 0) ok = bounded_wait(&ss->tmem_full[acc], aph, p, ss);
    if (ptx::bar_red_or(kEpiBarrier, 32 * kNumEpiWarps, !ok)) break;
    ptx::tc_fence_after();
    const uint32_t tbase = ss->tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) +
                           static_cast<uint32_t>(acc * kTileN);
    const int f = q.f0 + static_cast<int>(rank) * kTileM + quarter * 32 + (lane & ~1);
    for (int c = half * 16; c < q.cols; c += 32) {
      float v[16];
      ptx::tmem_ld_32x32b_x16(tbase + c, v);
      uint16_t* out = static_cast<uint16_t*>(p.out) + static_cast<int64_t>(q.t0 + c + odd) * F + f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const __nv_bfloat162 mine = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
        const uint32_t m = *reinterpret_cast<const uint32_t*>(&mine);
        const uint32_t o = __shfl_xor_sync(0xFFFFFFFFu, m, 1);
        // even lanes: the first token of both lanes; odd lanes: the second
        const uint32_t st = odd ? __byte_perm(o, m, 0x7632) : __byte_perm(m, o, 0x5410);
        if (q.t0 + c + 2 * j + odd < q.tend && f < p.F) *reinterpret_cast<uint32_t*>(out + 2 * j * F) = st;
      }
    }
    ptx::tc_fence_before();
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive_cluster_tmem(empty0 + static_cast<uint32_t>(acc) * 8u);
  }
  // rows of no group: before the first and after the last
  const int64_t vec = F / 8, first = g.off[0] * vec, last = g.off[p.groups] * vec, all = p.T * vec;
  uint4* out = static_cast<uint4*>(p.out);
  const int64_t at = static_cast<int64_t>(blockIdx.x) * (32 * kNumEpiWarps) + (warp - 2) * 32 + lane;
  const int64_t step = static_cast<int64_t>(gridDim.x) * (32 * kNumEpiWarps);
  for (int64_t i = at; i < first; i += step) out[i] = make_uint4(0, 0, 0, 0);
  for (int64_t i = last + at; i < all; i += step) out[i] = make_uint4(0, 0, 0, 0);
}

struct GroupedMaps {
  CUtensorMap tok[4];
};

template <bool DGRAD>
__global__ void __launch_bounds__(kGThreads, 1)
    grouped_kernel(const __grid_constant__ CUtensorMap mapW, const __grid_constant__ GroupedMaps maps,
                   const GroupedParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* smA = smem;
  uint8_t* smB = smem + kGStages * kGA;
  SharedState* ss = reinterpret_cast<SharedState*>(smB + kGStages * kGB);
  GroupTable& g = *reinterpret_cast<GroupTable*>(reinterpret_cast<uint8_t*>(ss) + 512);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = ptx::cluster_ctarank();
  ptx::grid_dep_launch();  // the step that may follow starts as this grid's CTAs end
  if (threadIdx.x == 0) {
    for (int s = 0; s < kGStages; ++s) {
      ptx::mbar_init(&ss->full[s], 1);
      ptx::mbar_init(&ss->empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      ptx::mbar_init(&ss->tmem_full[a], 1);
      ptx::mbar_init(&ss->tmem_empty[a], 2 * kNumEpiWarps);
    }
    ptx::mbar_init(&ss->mma_done, 1);
    ss->abort = 0;
    ptx::fence_mbar_init();
    ptx::prefetch_tensormap(&mapW);
  }
  if (warp == 1) {
    __syncwarp();
    ptx::tmem_alloc_pair(&ss->tmem_base, kTmemCols);
    ptx::tmem_relinquish_pair();
  }
  __syncwarp();
  build_groups(p, g);
  ptx::tc_fence_before();
  __syncthreads();
  ptx::cluster_sync();
  ptx::tc_fence_after();
  if (warp == 0) {
    if (lane == 0) grouped_producer<DGRAD>(&mapW, maps.tok, p, g, smA, smB, ss, rank);
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) grouped_mma<DGRAD>(p, g, smA, smB, ss);
  } else {
    grouped_epilogue(p, g, ss, warp, lane, rank);
  }
  __syncwarp();
  ptx::tc_fence_before();
  __syncthreads();
  ptx::cluster_sync();
  if (warp == 1) {
    __syncwarp();
    ptx::tc_fence_after();
    ptx::tmem_dealloc_pair(ss->tmem_base, kTmemCols);
  }
}

// ---------------------------------------------------------------- few tokens

// The forward product of a few rows (decoding): every live expert's weights are
// read once for a handful of tokens, so the floor is that read, and what
// matters is to spread it evenly over the GPU and keep it streaming.  The
// 256-feature tiles above do neither (12 live experts of 2048 features are 96
// of them for 76 pairs).  Here a block takes 16 features of one expert; its
// eight warps share K (32 columns each in turn, so that a block reads 512
// contiguous bytes of a row at a time), multiply on the 16 x 8 x 16 warp-level
// matrix instruction, which takes its weights from registers (each is used
// once: staging it through shared memory for a larger instruction would only
// lengthen its way), and add their sums in shared memory in warp order.
// The instruction's k order is free as long as both operands agree: a lane
// loads 16 contiguous bytes (eight k) of its row and of its token, and feeds
// them to two instructions.  How far the loads run ahead (AHEAD) goes by how
// many blocks have work: with more than two an SM, two turns (fewer registers,
// more blocks an SM: 16 rows over 12 of 16 experts of 2048 x 4096 33 us in a
// graph, eight turns 35, four 36, one 41), with fewer, eight (one row: 7.2 us, two
// turns 8.3).
constexpr int kFewRows = 16, kFewWarps = 8, kFewTiles = 4;  // up to 4 x 8 tokens a pass

__device__ __forceinline__ uint4 ld_once(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

__device__ __forceinline__ void mma_16x8x16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                            uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Features f0 .. f0 + 15 (those below F) of tokens t0 .. t0 + 8 NT - 1 (those
// below tend), by the whole block.  Rows and tokens past the end repeat the
// last one; their results are not stored.
template <int NT, int AHEAD>
__device__ __forceinline__ void few_product(const uint16_t* W, const uint16_t* X, const GroupedParams& p, int f0, int t0,
                                            int tend, int K, float* s_sum) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  const int V = K >> 3;
  const uint4* w0 = reinterpret_cast<const uint4*>(W + static_cast<int64_t>(min(f0 + g, p.F - 1)) * K);
  const uint4* w1 = reinterpret_cast<const uint4*>(W + static_cast<int64_t>(min(f0 + g + 8, p.F - 1)) * K);
  const uint4* x[NT];
  float acc[NT][4];
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    x[i] = reinterpret_cast<const uint4*>(X + static_cast<int64_t>(min(t0 + 8 * i + g, tend - 1)) * K);
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
  }
  const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll AHEAD
  for (int v = warp * 4 + q; v - q < V; v += kFewWarps * 4) {  // uniform over the warp
    const bool in = v < V;
    const uint4 a = in ? ld_once(w0 + v) : zero, b = in ? ld_once(w1 + v) : zero;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const uint4 t = in ? x[i][v] : zero;
      mma_16x8x16(acc[i], a.x, b.x, a.y, b.y, t.x, t.y);
      mma_16x8x16(acc[i], a.z, b.z, a.w, b.w, t.z, t.w);
    }
  }
  // [warp][token][feature]; a lane holds features g, g + 8 of tokens 2 q, 2 q + 1 of each tile
  constexpr int kCols = 8 * NT;
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
      s_sum[(warp * kCols + 8 * i + 2 * q + (j & 1)) * kFewRows + g + 8 * (j >> 1)] = acc[i][j];
  __syncthreads();
  for (int o = threadIdx.x; o < kCols * kFewRows; o += 32 * kFewWarps) {
    const int t = t0 + o / kFewRows, f = f0 + o % kFewRows;
    float sum = 0.f;
#pragma unroll
    for (int w = 0; w < kFewWarps; ++w) sum += s_sum[w * kCols * kFewRows + o];
    if (t < tend && f < p.F) {
      const __nv_bfloat16 b = __float2bfloat16_rn(sum);
      static_cast<uint16_t*>(p.out)[static_cast<int64_t>(t) * p.F + f] = *reinterpret_cast<const uint16_t*>(&b);
    }
  }
  __syncthreads();  // before the next pass overwrites the sums
}

template <int AHEAD>
__global__ void __launch_bounds__(32 * kFewWarps) grouped_few_kernel(const uint16_t* W, const uint16_t* X,
                                                                     const GroupedParams p, const int K) {
  __shared__ float s_sum[kFewWarps * 8 * kFewTiles * kFewRows];
  const int e = blockIdx.y, f0 = blockIdx.x * kFewRows;
  const int a = p.offsets[e], b = p.offsets[e + 1];
  // the table's rows (build_groups): each warp finds the largest offset up to e
  int most = 0;
  for (int i = threadIdx.x & 31; i <= e; i += 32) most = max(most, min(p.offsets[i], p.T));
  const int begin = __reduce_max_sync(0xFFFFFFFFu, most), end = max(begin, min(b, p.T));
  if (blockIdx.x == 0 && threadIdx.x == 0 && (a < 0 || b < a || b > p.T))
    atomicCAS(p.status, 0u, static_cast<uint32_t>(kStatusInvalid));
  const uint16_t* We = W + static_cast<int64_t>(e) * p.F * K;
  for (int t0 = begin; t0 < end; t0 += 8 * kFewTiles) {
    if (end - t0 <= 8) few_product<1, AHEAD>(We, X, p, f0, t0, end, K, s_sum);
    else if (end - t0 <= 16) few_product<2, AHEAD>(We, X, p, f0, t0, end, K, s_sum);
    else few_product<kFewTiles, AHEAD>(We, X, p, f0, t0, end, K, s_sum);
  }
  // rows of no group: before the first and after the last
  const int f = f0 + static_cast<int>(threadIdx.x);
  if (threadIdx.x < kFewRows && f < p.F) {
    uint16_t* Y = static_cast<uint16_t*>(p.out);
    if (e == 0)
      for (int t = 0; t < begin; ++t) Y[static_cast<int64_t>(t) * p.F + f] = 0;
    if (e == p.groups - 1)
      for (int t = end; t < p.T; ++t) Y[static_cast<int64_t>(t) * p.F + f] = 0;
  }
}

template <bool DGRAD>
cudaError_t run_grouped(const CUtensorMap& w, const GroupedMaps& m, const GroupedParams& p, int grid, cudaStream_t s) {
  auto* k = grouped_kernel<DGRAD>;
  const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kGSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
  cfg.blockDim = dim3(kGThreads, 1, 1);
  cfg.dynamicSmemBytes = kGSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k, w, m, p);
}

}  // namespace

cudaError_t launch_grouped_few(const void* W, const void* X, const GroupedParams& p, int K, int num_sms,
                               cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>((p.F + kFewRows - 1) / kFewRows), static_cast<unsigned>(p.groups));
  const auto* w = static_cast<const uint16_t*>(W);
  const auto* x = static_cast<const uint16_t*>(X);
  const int live = p.groups < p.T ? p.groups : p.T;  // groups with rows, at most
  if (static_cast<int64_t>(grid.x) * live > 2 * num_sms) grouped_few_kernel<2><<<grid, 32 * kFewWarps, 0, s>>>(w, x, p, K);
  else grouped_few_kernel<8><<<grid, 32 * kFewWarps, 0, s>>>(w, x, p, K);
  return cudaGetLastError();
}

cudaError_t launch_grouped(bool dgrad, const CUtensorMap& w, const CUtensorMap (&tok)[4],
                           const GroupedParams& p, int grid, cudaStream_t s) {
  GroupedMaps m;
  for (int i = 0; i < 4; ++i) m.tok[i] = tok[i];
  return dgrad ? run_grouped<true>(w, m, p, grid, s) : run_grouped<false>(w, m, p, grid, s);
}

}  // namespace forge
