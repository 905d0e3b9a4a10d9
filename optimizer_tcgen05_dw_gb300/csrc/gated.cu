// The gated feed-forward products.
//
// Forward, both projections of a token, the gate's activation and the product
// in one kernel:
//   G = X Wg^T,  U = X Wu^T,  Y = act(G) U          (W = [Wg; Wu], 2F x K)
// The pair's two CTAs hold the two halves of the matrix instruction's B
// operand, so one loads gate rows and the other up rows of the same features:
// every CTA's accumulator then has G in its first W columns and U in the next,
// and the activation meets its factor in one thread.  What the gradient needs
// (G and U) leaves in bf16 or as E4M3 codes; the 128 features of a tile are one
// block of the codes.
//
// Gradient, through the down projection's weight Wd [N x F], the product dY Wd
// with the activation's gradient as its epilogue (dA never reaches memory):
//   dA = dY Wd,  dU = dA act(G),  dG = dA U act'(G),  and Y = act(G) U again,
// which the down projection's own step reads: the forward need not keep it.
#include <cuda_bf16.h>

#include "codes.cuh"
#include "gate.cuh"
#include "pair_gemm.cuh"

namespace forge {

namespace {

constexpr int kQuarterBarrier = 2;  // + 0 .. 3: the four warps of a tensor-memory quarter

// ---------------------------------------------------------------- forward

template <int W, bool CODES, int AROWS = kTileM>
struct GatedOp {
  static_assert(!CODES || W == codes::kBlock, "a block of the codes is a tile's features");
  using Params = GatedParams;
  struct Maps { int unused; };
  static constexpr int kW = W, kARows = AROWS, kBufs = W == 128 ? 2 : 4, kSplit = 1;
  static constexpr int kStg = AROWS < kTileM ? (W == 128 ? 10 : W == 64 ? 16 : 24) : (W == 128 ? (CODES ? 5 : 6) : W == 64 ? 9 : 11);
  static constexpr int NC = W / 4;                            // features a warp takes
  static constexpr bool kRows = W == 128 && AROWS == kTileM;  // outputs meet in shared memory, to leave by rows
  static constexpr int kOut = kRows ? 32 * 32 * 2 : 0;        // a warp's bytes of it: 32 rows x 32 bf16
  static constexpr int kEpiBytes = pairs::kEpiWarps * kOut + (CODES ? 2 * 4 * kTileM * 4 : 0);
  static constexpr bool kMoreRegs = W == 128, kFp8 = false, kBMajorMN = false;
  // The tensor cores' sums are truncated, 1e-9 of a sum for each of its terms on
  // average: nothing beside bf16, but the scales of the codes are float32.  So
  // these are summed over 64 kFold terms at a time, and the sums in registers
  // (mean error of a scale at K = 5120: -5.0e-6 in one sum, -6.2e-7 so;
  // 4099 x 17408 tokens and features 800 us either way, 838 with kFold = 8: the
  // tensor cores then wait for the outputs of the tile before).
  static constexpr int kFold = CODES ? 12 : 0;

  // rank 0: gate rows, rank 1: up rows of the same features (rows of another
  // half past a ragged end give columns that are not stored)
  static __device__ __forceinline__ int b_row(int tn, int rank, const Params& p) { return rank * p.F + tn * W; }

  static __device__ __forceinline__ void init_barriers(pairs::Shared*) {}
  static __device__ __forceinline__ void helper(const Params&, pairs::Shared*, uint8_t*, int, int, uint32_t) {}

  static __device__ __forceinline__ void epilogue(const Maps&, const Params& p, pairs::Shared* ss, uint8_t* epi, int warp,
                                                  int lane, uint32_t rank) {
    const int quarter = warp & 3, sub = (warp - pairs::kFirstEpiWarp) >> 2, r = quarter * 32 + lane;
    const uint32_t empty0 = ptx::mapa(ptx::smem_addr(&ss->tmem_empty[0]), 0);
    float* red = reinterpret_cast<float*>(epi + pairs::kEpiWarps * kOut);  // [gate, up][warp of the quarter][row]
    uint8_t* out = epi + (warp - pairs::kFirstEpiWarp) * kOut;
    uint32_t acc = 0, ph = 0;
    for (int tile = pair_id(); tile < p.num_tiles; tile += num_pairs()) {
      int tm, tn;
      tile_coords_of(tile, p.tiles_m, p.tiles_n, tm, tn);
      const int64_t row = static_cast<int64_t>(tm) * kPairM + static_cast<int>(rank) * kTileM + r;
      const int f0 = tn * W + sub * NC;
      float g[NC], u[NC];
      // Hands the accumulator on after reading columns of it with `take`.
      auto read = [&](auto&& take) -> bool {
        if (!pairs::warp_wait(&ss->tmem_full[acc], ph, p, ss, lane)) return false;
        ptx::tc_fence_after();
        take(ss->tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + acc * (kTmemCols / kBufs) +
             static_cast<uint32_t>(sub * NC));
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive_cluster_tmem(empty0 + acc * 8u);
        if (++acc == kBufs) {
          acc = 0;
          ph ^= 1u;
        }
        return true;
      };
      bool ok = read([&](uint32_t at) {
        pairs::tmem_load<NC>(at, g);
        pairs::tmem_load<NC>(at + W, u);
      });
      if constexpr (CODES) {
        for (int kb = kFold; ok && kb < p.num_kb; kb += kFold)
          ok = read([&](uint32_t at) {
            float v[NC];
            pairs::tmem_load<NC>(at, v);
#pragma unroll
            for (int j = 0; j < NC; ++j) g[j] += v[j];
            pairs::tmem_load<NC>(at + W, v);
#pragma unroll
            for (int j = 0; j < NC; ++j) u[j] += v[j];
          });
        if (ptx::bar_red_or(kQuarterBarrier + quarter, 128, !ok)) return;  // the quarter's warps meet below: they stop together
        __syncwarp();
      } else if (!ok) {
        return;
      }
      float gs = 0.f, us = 0.f;
      if (CODES) {
        float ga = 0.f, ua = 0.f;
#pragma unroll
        for (int j = 0; j < NC; ++j) {  // (columns past F are of other rows)
          if (f0 + j < p.F) {
            ga = codes::max_nan(ga, fabsf(g[j]));
            ua = codes::max_nan(ua, fabsf(u[j]));
          }
        }
        red[sub * kTileM + r] = ga;
        red[(4 + sub) * kTileM + r] = ua;
        ptx::bar_sync(kQuarterBarrier + quarter, 128);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          ga = codes::max_nan(ga, red[i * kTileM + r]);
          ua = codes::max_nan(ua, red[(4 + i) * kTileM + r]);
        }
        gs = codes::block_scale(ga);
        us = codes::block_scale(ua);
        // (the next tile's first barrier keeps its sums from overtaking these reads)
      }
      if constexpr (CODES) {
        if (sub < 2 && row < p.T) p.scale[(row * 2 + sub) * p.tiles_n + tn] = sub == 0 ? gs : us;
      }
      if constexpr (kRows) {
        const int row0 = tm * kPairM + static_cast<int>(rank) * kTileM + quarter * 32;
        if (row0 >= p.T || f0 >= p.F) continue;
        if (p.gu != nullptr) {
          store_rows(out, g, static_cast<uint16_t*>(p.gu), int64_t{2} * p.F, p, row0, f0, lane);
          store_rows(out, u, static_cast<uint16_t*>(p.gu) + p.F, int64_t{2} * p.F, p, row0, f0, lane);
        }
        if constexpr (CODES)
          store_codes(out, g, u, codes::inverse_scale(gs), codes::inverse_scale(us), p, row0, f0, lane);
        gate(p.act, g, u);
        store_rows(out, g, static_cast<uint16_t*>(p.Y), p.F, p, row0, f0, lane);
      } else if (row < p.T) {
        if (p.gu != nullptr) {
          uint16_t* kept = static_cast<uint16_t*>(p.gu) + row * 2 * p.F + f0;
#pragma unroll
          for (int j = 0; j < NC / 8; ++j) {
            if (f0 + 8 * j >= p.F) break;
            *reinterpret_cast<uint4*>(kept + 8 * j) = pack_rne_bf16x8(reinterpret_cast<const float(&)[8]>(g[8 * j]));
            *reinterpret_cast<uint4*>(kept + p.F + 8 * j) = pack_rne_bf16x8(reinterpret_cast<const float(&)[8]>(u[8 * j]));
          }
        }
        gate(p.act, g, u);
        uint16_t* to = static_cast<uint16_t*>(p.Y) + row * p.F + f0;
#pragma unroll
        for (int j = 0; j < NC / 8; ++j) {
          if (f0 + 8 * j >= p.F) break;
          *reinterpret_cast<uint4*>(to + 8 * j) = pack_rne_bf16x8(reinterpret_cast<const float(&)[8]>(g[8 * j]));
        }
      }
    }
  }

  // Y over G.
  static __device__ __forceinline__ void gate(int act, float (&g)[NC], const float (&u)[NC]) {
    if (act == kActSilu) {
#pragma unroll
      for (int j = 0; j < NC; ++j) g[j] = gated<kActSilu>(g[j], u[j]);
    } else {
#pragma unroll
      for (int j = 0; j < NC; ++j) g[j] = gated<kActGeluTanh>(g[j], u[j]);
    }
  }

  // 32 rows x 32 features, a row a lane, to memory four lanes a row: 64
  // contiguous bytes of eight rows a store, where a lane's own row would be one
  // of 32 lines (16384 x 14336 with gu kept: 2419 us so, 2300 this way).
  static __device__ __forceinline__ void store_rows(uint8_t* buf, const float* v, uint16_t* to, int64_t ld, const Params& p,
                                                    int row0, int f0, int lane) {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      *reinterpret_cast<uint4*>(buf + sw64(lane, q)) = pack_rne_bf16x8(reinterpret_cast<const float(&)[8]>(v[8 * q]));
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 8 * i + (lane >> 2), q = lane & 3;
      if (row0 + r < p.T && f0 + 8 * q < p.F)
        *reinterpret_cast<uint4*>(to + (row0 + r) * ld + f0 + 8 * q) = *reinterpret_cast<const uint4*>(buf + sw64(r, q));
    }
    __syncwarp();
  }
  // The codes of G and U likewise: 32 bytes of each a row.
  static __device__ __forceinline__ void store_codes(uint8_t* buf, const float* g, const float* u, float gi, float ui,
                                                     const Params& p, int row0, int f0, int lane) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float* v = (q < 2 ? g : u) + 16 * (q & 1);
      const float k = q < 2 ? gi : ui;
      *reinterpret_cast<uint4*>(buf + sw64(lane, q)) =
          make_uint4(codes::encode4(v[0] * k, v[1] * k, v[2] * k, v[3] * k), codes::encode4(v[4] * k, v[5] * k, v[6] * k, v[7] * k),
                     codes::encode4(v[8] * k, v[9] * k, v[10] * k, v[11] * k),
                     codes::encode4(v[12] * k, v[13] * k, v[14] * k, v[15] * k));
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 8 * i + (lane >> 2), q = lane & 3, f = f0 + 16 * (q & 1);
      if (row0 + r < p.T && f < p.F) {  // (F % 8 == 0: eight codes at a time)
        uint8_t* to = static_cast<uint8_t*>(p.codes) + (static_cast<int64_t>(row0 + r) * 2 + (q >> 1)) * p.F + f;
        const uint4 c = *reinterpret_cast<const uint4*>(buf + sw64(r, q));
        *reinterpret_cast<uint2*>(to) = make_uint2(c.x, c.y);
        if (f + 8 < p.F) *reinterpret_cast<uint2*>(to + 8) = make_uint2(c.z, c.w);
      }
    }
    __syncwarp();
  }
};

// ---------------------------------------------------------------- gradient

// A row is a lane of the accumulator, so direct accesses would touch 32 lines an
// instruction (16384 x 14336 through 4096: 1946 us so).  What was kept comes in
// and dG, dU and Y go out four lanes a row, 64 contiguous bytes of eight rows an
// instruction, and every warp turns its own 32 rows x 32 features between the two
// in 2 KB of shared memory, one tensor after the other.  Copies of the
// tensor-memory accelerator would turn them too, but they take its time from the
// operands', and larger buffers, which the ring is better used for (what was kept
// by copies, 6 KB a warp and 4 stages: 1318 us; 4 KB and 5 stages: 1240; so, 6
// stages: 1146, the products alone 969).
// A warp's first chunk of a tile is loaded before its products are there, and the
// other asked into L2 (in registers there is no room for it: the spills of that
// cost more, 1372 us).
template <int W, bool CODES>
struct GatedGradOp {
  using Params = GatedParams;
  struct Maps { int unused; };
  static constexpr int kW = W, kARows = kTileM, kStg = W == 128 ? 6 : 8, kBufs = W == 128 ? 2 : 4, kSplit = 1;
  static constexpr int NC = W / 2, kChunk = 32;        // features a warp takes, and at a time
  static constexpr int kTurn = 32 * kChunk * 2;        // bytes of a chunk of one tensor in bf16
  static constexpr int kLoads = CODES ? 4 : 8;         // 16-byte vectors a lane loads of a chunk
  static constexpr int kEpiBytes = pairs::kEpiWarps * kTurn;
  static constexpr bool kMoreRegs = false, kFp8 = false, kBMajorMN = true;
  static constexpr int kFold = 0;

  static __device__ __forceinline__ int b_row(int tn, int rank, const Params&) { return (2 * tn + rank) * W; }
  static __device__ __forceinline__ void init_barriers(pairs::Shared*) {}
  static __device__ __forceinline__ void helper(const Params&, pairs::Shared*, uint8_t*, int, int, uint32_t) {}

  // This lane's vectors of what was kept for the chunk at (row0, f): of rows
  // 8 i + lane / 4, eight features of G (vectors 0-3) and of U (4-7); or in codes
  // sixteen, of G in its even lanes' pairs and of U in the others'.
  static __device__ __forceinline__ void load(uint4 (&v)[kLoads], const Params& p, int row0, int f, int lane) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = row0 + 8 * i + (lane >> 2), q = lane & 3;
      v[i] = make_uint4(0, 0, 0, 0);
      if constexpr (CODES) {
        const int at = f + 16 * (q & 1);
        const uint8_t* from = static_cast<const uint8_t*>(p.codes) + (static_cast<int64_t>(r) * 2 + (q >> 1)) * p.F + at;
        if (r < p.T && at < p.F) {  // (F % 8 == 0: eight codes at a time)
          const uint2 a = __ldcs(reinterpret_cast<const uint2*>(from));
          v[i].x = a.x;
          v[i].y = a.y;
        }
        if (r < p.T && at + 8 < p.F) {
          const uint2 a = __ldcs(reinterpret_cast<const uint2*>(from + 8));
          v[i].z = a.x;
          v[i].w = a.y;
        }
      } else {
        v[i + 4] = v[i];
        if (r < p.T && f + 8 * q < p.F) {
          const uint16_t* from = static_cast<const uint16_t*>(p.gu) + static_cast<int64_t>(r) * 2 * p.F + f + 8 * q;
          v[i] = __ldcs(reinterpret_cast<const uint4*>(from));
          v[i + 4] = __ldcs(reinterpret_cast<const uint4*>(from + p.F));
        }
      }
    }
  }
  static __device__ __forceinline__ void prefetch_l2(const void* at) { asm volatile("prefetch.global.L2 [%0];" ::"l"(at)); }
  // 32 rows of four vectors: from four lanes a row to a row a lane.
  static __device__ __forceinline__ void turn(uint8_t* buf, const uint4* in, uint4* out, int lane) {
#pragma unroll
    for (int i = 0; i < 4; ++i) *reinterpret_cast<uint4*>(buf + sw64(8 * i + (lane >> 2), lane & 3)) = in[i];
    __syncwarp();
#pragma unroll
    for (int q = 0; q < 4; ++q) out[q] = *reinterpret_cast<const uint4*>(buf + sw64(lane, q));
    __syncwarp();
  }
  // And back, to memory: rows of `to`, ld elements apart.
  static __device__ __forceinline__ void store(uint8_t* buf, const uint4* v, uint16_t* to, int64_t ld, const Params& p, int row0,
                                               int f, int lane, uint64_t pol) {
#pragma unroll
    for (int q = 0; q < 4; ++q) *reinterpret_cast<uint4*>(buf + sw64(lane, q)) = v[q];
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 8 * i + (lane >> 2), q = lane & 3;
      if (row0 + r < p.T && f + 8 * q < p.F)
        st_stream(to + (row0 + r) * ld + f + 8 * q, *reinterpret_cast<const uint4*>(buf + sw64(r, q)), pol);
    }
    __syncwarp();
  }

  static __device__ __forceinline__ void epilogue(const Maps&, const Params& p, pairs::Shared* ss, uint8_t* epi, int warp,
                                                  int lane, uint32_t rank) {
    const int quarter = warp & 3, w = warp - pairs::kFirstEpiWarp, sub = w >> 2;
    const uint32_t empty0 = ptx::mapa(ptx::smem_addr(&ss->tmem_empty[0]), 0);
    const int NB = (p.F + codes::kBlock - 1) / codes::kBlock;
    uint8_t* buf = epi + w * kTurn;
    const uint64_t pol = evict_first_policy();  // (what streams through should not displace the operands in L2)
    uint32_t acc = 0, ph = 0;
    for (int tile = pair_id(); tile < p.num_tiles; tile += num_pairs()) {
      int tm, tn;
      tile_coords_of(tile, p.tiles_m, p.tiles_n, tm, tn);
      const int row0 = tm * kPairM + static_cast<int>(rank) * kTileM + quarter * 32, f0 = tn * 2 * W + sub * NC;
      const int64_t row = row0 + lane;
      const uint32_t taddr = ss->tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + acc * (kTmemCols / kBufs) +
                             static_cast<uint32_t>(sub * NC);
      bool ready = false;  // the accumulator is
#pragma unroll 1
      for (int f = f0; f < f0 + NC && row0 < p.T && f < p.F; f += kChunk) {
        float gs = 0.f, us = 0.f;
        if (CODES && row < p.T) {
          gs = p.scale[row * 2 * NB + f / codes::kBlock];
          us = p.scale[(row * 2 + 1) * NB + f / codes::kBlock];
        }
        uint4 kept[kLoads], rows[kLoads];
        load(kept, p, row0, f, lane);
        if (!ready) {
          if (row < p.T && f + kChunk < min(f0 + NC, p.F)) {
            const int64_t at = row * 2 * p.F + f + kChunk;
            if (CODES) {
              prefetch_l2(static_cast<const uint8_t*>(p.codes) + at);
              prefetch_l2(static_cast<const uint8_t*>(p.codes) + at + p.F);
            } else {
              prefetch_l2(static_cast<const uint16_t*>(p.gu) + at);
              prefetch_l2(static_cast<const uint16_t*>(p.gu) + at + p.F);
            }
          }
          if (!pairs::warp_wait(&ss->tmem_full[acc], ph, p, ss, lane)) return;
          ptx::tc_fence_after();
          ready = true;
        }
#pragma unroll
        for (int i = 0; i < kLoads; i += 4) turn(buf, kept + i, rows + i, lane);
        float da[kChunk];
        pairs::tmem_load<kChunk>(taddr + (f - f0), da);
        uint4 dg[4], du[4], y[4];
        if (p.act == kActSilu) gradients<kActSilu>(da, rows, gs, us, dg, du, y);
        else gradients<kActGeluTanh>(da, rows, gs, us, dg, du, y);
        store(buf, dg, static_cast<uint16_t*>(p.dGU), int64_t{2} * p.F, p, row0, f, lane, pol);
        store(buf, du, static_cast<uint16_t*>(p.dGU) + p.F, int64_t{2} * p.F, p, row0, f, lane, pol);
        if (p.Y != nullptr) store(buf, y, static_cast<uint16_t*>(p.Y), p.F, p, row0, f, lane, pol);
      }
      if (!ready && !pairs::warp_wait(&ss->tmem_full[acc], ph, p, ss, lane)) return;  // nothing of it is this warp's
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive_cluster_tmem(empty0 + acc * 8u);
      if (++acc == kBufs) {
        acc = 0;
        ph ^= 1u;
      }
    }
  }

  // A lane's 32 features, G in the first half of `rows` and U in the second: dG, dU and Y.
  template <int ACT>
  static __device__ __forceinline__ void gradients(const float (&da)[kChunk], const uint4 (&rows)[kLoads], float gs, float us,
                                                   uint4 (&dg)[4], uint4 (&du)[4], uint4 (&out)[4]) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      float g[8], u[8], y[8];
      if constexpr (CODES) {
        const uint4 a = rows[q >> 1], b = rows[2 + (q >> 1)];
        decode8(q & 1 ? make_uint2(a.z, a.w) : make_uint2(a.x, a.y), gs, g);
        decode8(q & 1 ? make_uint2(b.z, b.w) : make_uint2(b.x, b.y), us, u);
      } else {
        unpack_bf16x8(rows[q], g);
        unpack_bf16x8(rows[4 + q], u);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) gated_gradient<ACT>(da[8 * q + j], g[j], u[j], g[j], u[j], y[j]);
      dg[q] = pack_rne_bf16x8(g);
      du[q] = pack_rne_bf16x8(u);
      out[q] = pack_rne_bf16x8(y);
    }
  }

  static __device__ __forceinline__ void decode8(uint2 c, float scale, float (&v)[8]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 d = codes::decode2((j < 2 ? c.x : c.y) >> (16 * (j & 1)));
      v[2 * j] = d.x * scale;
      v[2 * j + 1] = d.y * scale;
    }
  }
};

}  // namespace

cudaError_t launch_gated(int width, const CUtensorMap& x, const CUtensorMap& w, const GatedParams& p, int pairs_n,
                         cudaStream_t s) {
  if (p.codes != nullptr) return pairs::launch<GatedOp<128, true>>(x, w, {}, p, pairs_n, s);
  if (p.T <= kShortRows) {
    if (width == 128) return pairs::launch<GatedOp<128, false, kShortRows>>(x, w, {}, p, pairs_n, s);
    if (width == 64) return pairs::launch<GatedOp<64, false, kShortRows>>(x, w, {}, p, pairs_n, s);
    return pairs::launch<GatedOp<32, false, kShortRows>>(x, w, {}, p, pairs_n, s);
  }
  if (width == 128) return pairs::launch<GatedOp<128, false>>(x, w, {}, p, pairs_n, s);
  if (width == 64) return pairs::launch<GatedOp<64, false>>(x, w, {}, p, pairs_n, s);
  return pairs::launch<GatedOp<32, false>>(x, w, {}, p, pairs_n, s);
}

template <int W>
static cudaError_t run_grad(const CUtensorMap& dy, const CUtensorMap& w, const GatedParams& p, int pairs_n, cudaStream_t s) {
  if (p.codes == nullptr) return pairs::launch<GatedGradOp<W, false>>(dy, w, {}, p, pairs_n, s);
  return pairs::launch<GatedGradOp<W, true>>(dy, w, {}, p, pairs_n, s);
}

cudaError_t launch_gated_grad(int width, const CUtensorMap& dy, const CUtensorMap& w, const GatedParams& p, int pairs_n,
                              cudaStream_t s) {
  return width == 128 ? run_grad<128>(dy, w, p, pairs_n, s) : run_grad<64>(dy, w, p, pairs_n, s);
}

}  // namespace forge
