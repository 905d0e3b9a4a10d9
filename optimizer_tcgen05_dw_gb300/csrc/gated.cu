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

// Byte offset of 16-byte chunk c of row r in a box of 32-byte rows stored with the 32-byte swizzle.
__device__ __forceinline__ uint32_t sw32(int r, int c) { return static_cast<uint32_t>(r * 32 + ((c ^ ((r >> 2) & 1)) << 4)); }

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
  static constexpr bool kMoreRegs = W == 128, kFp8 = false, kBMajorMN = false, kBlockwise = false;

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
      const bool ok = pairs::warp_wait(&ss->tmem_full[acc], ph, p, ss, lane);
      if (CODES) {  // the quarter's warps meet below: they stop together
        if (ptx::bar_red_or(kQuarterBarrier + quarter, 128, !ok)) return;
        __syncwarp();
      } else if (!ok) {
        return;
      }
      ptx::tc_fence_after();
      const uint32_t taddr = ss->tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + acc * (kTmemCols / kBufs) +
                             static_cast<uint32_t>(sub * NC);
      float g[NC], u[NC];
      pairs::tmem_load<NC>(taddr, g);
      pairs::tmem_load<NC>(taddr + W, u);
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive_cluster_tmem(empty0 + acc * 8u);
      if (++acc == kBufs) {
        acc = 0;
        ph ^= 1u;
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

// What was kept is read and dGU and Y are written through shared memory, chunk
// by chunk, every warp its own 32 rows x 32 features: a row is a lane, so direct
// accesses would touch 32 lines an instruction (16384 x 14336 through 4096: 1946 us
// so).  In, copies of the tensor-memory accelerator bring a chunk's G and U; a
// warp's first chunk of a tile comes while the tile's products are formed.  dG and dU replace what they came from and go out
// by ordinary stores, four lanes a row: as copies of the accelerator, whose rows
// are of 64 bytes, they took its time from the operands' (1455 us; the products
// alone 969).  Codes with F % 16 != 0, whose rows the accelerator cannot address,
// are loaded directly (VIA false).
template <int W, bool CODES, bool VIA>
struct GatedGradOp {
  using Params = GatedParams;
  struct Maps { CUtensorMap kept; };
  static constexpr int kW = W, kARows = kTileM, kStg = W == 128 ? 4 : 5, kBufs = W == 128 ? 2 : 4, kSplit = 1;
  static constexpr int NC = W / 2, kChunk = 32;        // features a warp takes, and at a time
  static constexpr int kPair = 32 * 2 * kChunk * 2;    // bytes of a chunk of dG and dU (and of G and U in bf16)
  static constexpr int kOne = 32 * kChunk * 2;         // of Y (and of G's and U's codes together)
  static constexpr int kEpiBytes = pairs::kEpiWarps * (kPair + kOne);
  static constexpr bool kMoreRegs = false, kFp8 = false, kBMajorMN = true, kBlockwise = false;

  static __device__ __forceinline__ int b_row(int tn, int rank, const Params&) { return (2 * tn + rank) * W; }
  static __device__ __forceinline__ void init_barriers(pairs::Shared* ss) {
    for (int i = 0; i < pairs::kEpiWarps; ++i) ptx::mbar_init(&ss->epi[i], 1);
  }
  static __device__ __forceinline__ void helper(const Params&, pairs::Shared*, uint8_t*, int, int, uint32_t) {}

  static __device__ __forceinline__ void epilogue(const Maps& maps, const Params& p, pairs::Shared* ss, uint8_t* epi,
                                                  int warp, int lane, uint32_t rank) {
    const int quarter = warp & 3, w = warp - pairs::kFirstEpiWarp, sub = w >> 2;
    const uint32_t empty0 = ptx::mapa(ptx::smem_addr(&ss->tmem_empty[0]), 0);
    const int NB = (p.F + codes::kBlock - 1) / codes::kBlock;
    // A lane computes its own row's bytes of each alone.
    uint8_t* both = epi + w * (kPair + kOne);  // [gate, up][row][32] bf16, 64-byte swizzle
    uint8_t* one = both + kPair;               // [row][32] bf16, 64-byte swizzle; or codes [gate, up][row][32], 32-byte swizzle
    uint64_t* bar = &ss->epi[w];
    const uint64_t pol = evict_first_policy();  // (what streams through should not displace the operands in L2)
    uint32_t acc = 0, ph = 0, kept_ph = 0;
    auto origin = [&](int tile, int& row0, int& f0) {
      int tm, tn;
      tile_coords_of(tile, p.tiles_m, p.tiles_n, tm, tn);
      row0 = tm * kPairM + static_cast<int>(rank) * kTileM + quarter * 32;
      f0 = tn * 2 * W + sub * NC;
    };
    // Begins the load of what was kept for the chunk at (row0, f); whether there is any of it.
    auto load = [&](int row0, int f) -> bool {
      const bool any = row0 < p.T && f < p.F;
      if (VIA && any && lane == 0) {
        ptx::mbar_arrive_expect_tx(bar, CODES ? kOne : kPair);
        uint8_t* to = CODES ? one : both;
        ptx::tma_load_3d(&maps.kept, bar, to, f, 0, row0);
        ptx::tma_load_3d(&maps.kept, bar, to + (CODES ? kOne : kPair) / 2, f, 1, row0);
      }
      return VIA && any;
    };
    bool loaded = false;  // a load is under way
    for (int tile = pair_id(); tile < p.num_tiles; tile += num_pairs()) {
      int row0, f0;
      origin(tile, row0, f0);
      if (!loaded) loaded = load(row0, f0);
      if (!pairs::warp_wait(&ss->tmem_full[acc], ph, p, ss, lane)) break;
      ptx::tc_fence_after();
      const uint32_t taddr = ss->tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + acc * (kTmemCols / kBufs) +
                             static_cast<uint32_t>(sub * NC);
      const int64_t row = row0 + lane;
      bool ok = true;
#pragma unroll 1
      for (int c = 0; c < NC && row0 < p.T && f0 + c < p.F; c += kChunk) {
        const int f = f0 + c;
        float gs = 0.f, us = 0.f;
        if (CODES && row < p.T) {
          gs = p.scale[row * 2 * NB + f / codes::kBlock];
          us = p.scale[(row * 2 + 1) * NB + f / codes::kBlock];
        }
        uint4 gc[2], uc[2];  // CODES: this row's
        if (VIA) {
          if (!(ok = pairs::warp_wait(bar, kept_ph, p, ss, lane))) break;
          kept_ph ^= 1u;
          loaded = false;
          if (CODES) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              gc[h] = *reinterpret_cast<const uint4*>(one + sw32(lane, h));
              uc[h] = *reinterpret_cast<const uint4*>(one + kOne / 2 + sw32(lane, h));
            }
            __syncwarp();  // before Y goes over them
          }
        } else {
#pragma unroll
          for (int h = 0; h < 4; ++h) {
            uint2 a = make_uint2(0, 0), b = a;
            if (row < p.T && f + 8 * h < p.F) {
              const uint8_t* at = static_cast<const uint8_t*>(p.codes) + row * 2 * p.F + f + 8 * h;
              a = *reinterpret_cast<const uint2*>(at);
              b = *reinterpret_cast<const uint2*>(at + p.F);
            }
            (h & 1 ? gc[h >> 1].z : gc[h >> 1].x) = a.x;
            (h & 1 ? gc[h >> 1].w : gc[h >> 1].y) = a.y;
            (h & 1 ? uc[h >> 1].z : uc[h >> 1].x) = b.x;
            (h & 1 ? uc[h >> 1].w : uc[h >> 1].y) = b.y;
          }
        }
        float da[kChunk];
        pairs::tmem_load<kChunk>(taddr + c, da);
        if (p.act == kActSilu) gradients<kActSilu>(da, gc, uc, gs, us, both, one, lane);
        else gradients<kActGeluTanh>(da, gc, uc, gs, us, both, one, lane);
        __syncwarp();
        // Out, four lanes a row: 64 contiguous bytes of eight rows a store.
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = 8 * i + (lane >> 2), q = lane & 3;
          if (row0 + r < p.T && f + 8 * q < p.F) {
            const int64_t at = static_cast<int64_t>(row0 + r) * 2 * p.F + f + 8 * q;
            uint16_t* out = static_cast<uint16_t*>(p.dGU) + at;
            st_stream(out, *reinterpret_cast<const uint4*>(both + sw64(r, q)), pol);
            st_stream(out + p.F, *reinterpret_cast<const uint4*>(both + kPair / 2 + sw64(r, q)), pol);
            if (p.Y != nullptr)
              st_stream(static_cast<uint16_t*>(p.Y) + static_cast<int64_t>(row0 + r) * p.F + f + 8 * q,
                        *reinterpret_cast<const uint4*>(one + sw64(r, q)), pol);
          }
        }
        ptx::fence_proxy_async_smem();  // before a copy fills the buffers again
        __syncwarp();
        // The next chunk: this tile's, or else the next tile's first.
        int next_row = row0, next_f = f + kChunk;
        const bool more = c + kChunk < NC && next_f < p.F;
        if (!more && tile + num_pairs() < p.num_tiles) origin(tile + num_pairs(), next_row, next_f);
        if (more || tile + num_pairs() < p.num_tiles) loaded = load(next_row, next_f);
      }
      if (!ok) break;
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive_cluster_tmem(empty0 + acc * 8u);
      if (++acc == kBufs) {
        acc = 0;
        ph ^= 1u;
      }
    }
    if (loaded && lane == 0) pairs::wait(bar, kept_ph, p, ss, false);  // (a load begun before the block gave up)
    __syncwarp();
  }

  // A lane's 32 features: dG and dU over G and U, and Y.
  template <int ACT>
  static __device__ __forceinline__ void gradients(const float (&da)[kChunk], const uint4 (&gc)[2], const uint4 (&uc)[2], float gs,
                                                   float us, uint8_t* both, uint8_t* one, int lane) {
#pragma unroll
    for (int q = 0; q < kChunk / 8; ++q) {
      float g[8], u[8], y[8];
      if (CODES) {
        decode8(q & 1 ? make_uint2(gc[q >> 1].z, gc[q >> 1].w) : make_uint2(gc[q >> 1].x, gc[q >> 1].y), gs, g);
        decode8(q & 1 ? make_uint2(uc[q >> 1].z, uc[q >> 1].w) : make_uint2(uc[q >> 1].x, uc[q >> 1].y), us, u);
      } else {
        unpack_bf16x8(*reinterpret_cast<const uint4*>(both + sw64(lane, q)), g);
        unpack_bf16x8(*reinterpret_cast<const uint4*>(both + kPair / 2 + sw64(lane, q)), u);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) gated_gradient<ACT>(da[8 * q + j], g[j], u[j], g[j], u[j], y[j]);
      *reinterpret_cast<uint4*>(both + sw64(lane, q)) = pack_rne_bf16x8(g);
      *reinterpret_cast<uint4*>(both + kPair / 2 + sw64(lane, q)) = pack_rne_bf16x8(u);
      *reinterpret_cast<uint4*>(one + sw64(lane, q)) = pack_rne_bf16x8(y);
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
static cudaError_t run_grad(const CUtensorMap& dy, const CUtensorMap& w, const CUtensorMap& kept, const GatedParams& p,
                            int pairs_n, cudaStream_t s) {
  if (p.codes == nullptr) return pairs::launch<GatedGradOp<W, false, true>>(dy, w, {kept}, p, pairs_n, s);
  if (p.F % 16 == 0) return pairs::launch<GatedGradOp<W, true, true>>(dy, w, {kept}, p, pairs_n, s);
  return pairs::launch<GatedGradOp<W, true, false>>(dy, w, {kept}, p, pairs_n, s);
}

cudaError_t launch_gated_grad(int width, const CUtensorMap& dy, const CUtensorMap& w, const CUtensorMap& kept,
                              const GatedParams& p, int pairs_n, cudaStream_t s) {
  return width == 128 ? run_grad<128>(dy, w, kept, p, pairs_n, s) : run_grad<64>(dy, w, kept, p, pairs_n, s);
}

}  // namespace forge
