// One optimizer step over many tensors: norms, embeddings, biases, gates --
// the parameters whose gradients exist as tensors and that the fused linear
// step does not reach.
//
// Per element the arithmetic is optim.cuh's rule<KIND> (the sequence of the
// fused epilogue), so a tensor steps here exactly as a linear's weight does
// there.  The step reads and writes each element's weight and moments once
// and reads its gradient once: 28 B per element with everything in float32,
// 22 B with bf16 weights and gradients, 14 B with bf16 moments as well, 10.25
// to 16.25 B with INT8 moments.  That traffic is the floor.  The arithmetic
// (AdamW: a division, a square root and, for bf16 weights, an eighth of a
// Philox call per element) stays under it with float32 moments (239 M elements
// 830 us, 6.3 TB/s); with bf16 ones it shows (34 M: 89 us, 5.3 TB/s), and INT8
// moments are bound by their instructions.
//
// Many short tensors would cost a launch each, so one launch takes up to 480
// of them: their pointers travel in the kernel's parameters (no copy to the
// device, no table to keep, and a call can be captured in a CUDA graph), and
// a block finds its tensor by binary search over the tensors' first tiles.
#include "elem.cuh"
#include "launch.h"
#include "optim.cuh"

namespace forge {

namespace {

constexpr int kMultiThreads = 256;

enum GDtype { kGFp32 = 0, kGBf16 = 1 };

// Elements e0 .. e0 + cnt - 1 (cnt <= 8, e0 a multiple of 8) of a float32 or
// bf16 tensor; a tensor's ragged last group goes element by element.
__device__ __forceinline__ void load_f32(const void* base, int64_t e0, int cnt, float (&v)[8]) {
  const float* p = static_cast<const float*>(base) + e0;
  if (cnt == 8) {
    load8(p, v);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = j < cnt ? p[j] : 0.f;
  }
}
__device__ __forceinline__ void store_f32(void* base, int64_t e0, int cnt, const float (&v)[8]) {
  float* p = static_cast<float*>(base) + e0;
  if (cnt == 8) {
    store8(p, v);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < cnt) p[j] = v[j];
  }
}
__device__ __forceinline__ void load_b16(const void* base, int64_t e0, int cnt, float (&v)[8]) {
  if (cnt == 8) {
    load_bf16x8(base, e0, v);
  } else {
    const uint16_t* p = static_cast<const uint16_t*>(base) + e0;
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = j < cnt ? dev::bf16_to_f32(p[j]) : 0.f;
  }
}
// Eight bf16 values packed in pairs.
__device__ __forceinline__ void store_b16(void* base, int64_t e0, int cnt, uint4 v) {
  uint16_t* p = static_cast<uint16_t*>(base) + e0;
  if (cnt == 8) {
    *reinterpret_cast<uint4*>(p) = v;
  } else {
    const uint32_t a[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < cnt) p[j] = static_cast<uint16_t>(a[j >> 1] >> (16 * (j & 1)));
  }
}
template <bool SIGNED>
__device__ __forceinline__ void load_c8(const void* base, int64_t e0, int cnt, float a, float (&v)[8]) {
  const uint8_t* p = static_cast<const uint8_t*>(base) + e0;
  uint2 c = make_uint2(0u, 0u);
  if (cnt == 8) {
    c = *reinterpret_cast<const uint2*>(p);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < cnt) (j < 4 ? c.x : c.y) |= static_cast<uint32_t>(p[j]) << (8 * (j & 3));
  }
  decode8<SIGNED>(c, a, v);
}
template <bool SIGNED>
__device__ __forceinline__ void store_c8(void* base, int64_t e0, int cnt, float a, const float (&v)[8]) {
  uint8_t* p = static_cast<uint8_t*>(base) + e0;
  const uint2 c = encode8<SIGNED>(v, a);
  if (cnt == 8) {
    *reinterpret_cast<uint2*>(p) = c;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < cnt) p[j] = static_cast<uint8_t>((j < 4 ? c.x : c.y) >> (8 * (j & 3)));
  }
}

// One group of eight elements (cnt of them inside the tensor, none when the
// thread lies past its end).
template <int KIND, int WDT, int SDT, int GDT>
__device__ __forceinline__ void multi_group(const MultiItem& it, const OptScalars& sc, uint64_t seed,
                                            uint64_t step, int qblock, int64_t e0, int cnt) {
  float g[8], w[8], s1[8], s2[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) g[j] = w[j] = s1[j] = s2[j] = 0.f;
  const int64_t blk = SDT == kSInt8 ? e0 / qblock : 0;
  if (cnt > 0) {
    if (it.g != nullptr) {
      if (GDT == kGBf16) load_b16(it.g, e0, cnt, g);
      else load_f32(it.g, e0, cnt, g);
    }
    if (WDT == kWBf16) load_b16(it.W, e0, cnt, w);
    else load_f32(it.W, e0, cnt, w);
    if (SDT == kSInt8) {
      if (uses_s1(KIND)) load_c8<true>(it.s1, e0, cnt, it.s1_scale[blk], s1);
      if (uses_s2(KIND)) load_c8<false>(it.s2, e0, cnt, it.s2_scale[blk], s2);
    } else if (SDT == kSBf16) {
      if (uses_s1(KIND)) load_b16(it.s1, e0, cnt, s1);
      if (uses_s2(KIND)) load_b16(it.s2, e0, cnt, s2);
    } else {
      if (uses_s1(KIND)) load_f32(it.s1, e0, cnt, s1);
      if (uses_s2(KIND)) load_f32(it.s2, e0, cnt, s2);
    }
    dev::rule8<KIND>(w, g, s1, s2, sc);
    if (WDT == kWBf16) {
      store_b16(it.W, e0, cnt, pack_sr_bf16x8(w, dev::sr_words(static_cast<uint64_t>(e0) >> 3, seed + it.index, step)));
    } else {
      store_f32(it.W, e0, cnt, w);
    }
    if (SDT == kSFp32) {
      if (uses_s1(KIND)) store_f32(it.s1, e0, cnt, s1);
      if (uses_s2(KIND)) store_f32(it.s2, e0, cnt, s2);
    } else if (SDT == kSBf16) {
      if (uses_s1(KIND)) store_b16(it.s1, e0, cnt, pack_rne_bf16x8(s1));
      if (uses_s2(KIND)) store_b16(it.s2, e0, cnt, pack_rne_bf16x8(s2));
    }
  }
  if (SDT == kSInt8) {
    // the block's new absmax, over the qblock / 8 lanes that share it (a tile
    // holds whole blocks; elements past the tensor's end do not count)
    float n1 = 0.f, n2 = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      n1 = dev::absmax_acc(n1, j < cnt ? s1[j] : 0.f);
      n2 = dev::absmax_acc(n2, j < cnt ? s2[j] : 0.f);
    }
    if (uses_s1(KIND)) n1 = group_max(n1, qblock / 8);
    if (uses_s2(KIND)) n2 = group_max(n2, qblock / 8);
    if (cnt > 0) {
      const bool first = e0 == blk * qblock;
      if (uses_s1(KIND)) {
        store_c8<true>(it.s1, e0, cnt, n1, s1);
        if (first) it.s1_scale[blk] = n1;
      }
      if (uses_s2(KIND)) {
        store_c8<false>(it.s2, e0, cnt, n2, s2);
        if (first) it.s2_scale[blk] = n2;
      }
    }
  }
}

template <int WDT, int SDT, int GDT, int CAP>
__global__ void __launch_bounds__(kMultiThreads) multi_opt_kernel(const __grid_constant__ MultiParams<CAP> p) {
  // the last tensor whose first tile is not past this one
  int lo = 0, hi = p.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (p.items[mid].first <= blockIdx.x) lo = mid;
    else hi = mid - 1;
  }
  const MultiItem& it = p.items[lo];
  const int64_t e0 = static_cast<int64_t>(blockIdx.x - it.first) * kMultiTile + threadIdx.x * 8;
  const int64_t left = it.n - e0;
  const int cnt = left >= 8 ? 8 : (left > 0 ? static_cast<int>(left) : 0);
  switch (p.sc.kind) {
    case kAdamW: multi_group<kAdamW, WDT, SDT, GDT>(it, p.sc, p.seed, p.step, p.qblock, e0, cnt); break;
    case kNAdam: multi_group<kNAdam, WDT, SDT, GDT>(it, p.sc, p.seed, p.step, p.qblock, e0, cnt); break;
    case kRAdam: multi_group<kRAdam, WDT, SDT, GDT>(it, p.sc, p.seed, p.step, p.qblock, e0, cnt); break;
    case kLion: multi_group<kLion, WDT, SDT, GDT>(it, p.sc, p.seed, p.step, p.qblock, e0, cnt); break;
    case kRMSprop: multi_group<kRMSprop, WDT, SDT, GDT>(it, p.sc, p.seed, p.step, p.qblock, e0, cnt); break;
    case kAdaGrad: multi_group<kAdaGrad, WDT, SDT, GDT>(it, p.sc, p.seed, p.step, p.qblock, e0, cnt); break;
    case kSGD: multi_group<kSGD, WDT, SDT, GDT>(it, p.sc, p.seed, p.step, p.qblock, e0, cnt); break;
    default: multi_group<kSGDMomentum, WDT, SDT, GDT>(it, p.sc, p.seed, p.step, p.qblock, e0, cnt); break;
  }
}

template <int WDT, int SDT, int GDT, int CAP>
void run_multi_cap(const MultiParams<kMultiLong>& p, uint32_t tiles, cudaStream_t s) {
  MultiParams<CAP> q;
  q.sc = p.sc;
  q.seed = p.seed;
  q.step = p.step;
  q.count = p.count;
  q.qblock = p.qblock;
  for (int i = 0; i < p.count; ++i) q.items[i] = p.items[i];
  multi_opt_kernel<WDT, SDT, GDT, CAP><<<tiles, kMultiThreads, 0, s>>>(q);
}

// A launch costs host time for its parameters' bytes, so a table goes in the
// shortest of three forms that holds it (81 small tensors, a pass with the
// host's part: 7.2 us in 140 entries, 7.9 in 480).
template <int WDT, int SDT, int GDT>
cudaError_t run_multi(const MultiParams<kMultiLong>& p, uint32_t tiles, cudaStream_t s) {
  if (p.count <= kMultiShort) run_multi_cap<WDT, SDT, GDT, kMultiShort>(p, tiles, s);
  else if (p.count <= kMultiMiddle) run_multi_cap<WDT, SDT, GDT, kMultiMiddle>(p, tiles, s);
  else multi_opt_kernel<WDT, SDT, GDT, kMultiLong><<<tiles, kMultiThreads, 0, s>>>(p);
  return cudaGetLastError();
}

template <int WDT, int GDT>
cudaError_t run_multi_sdt(int sdt, const MultiParams<kMultiLong>& p, uint32_t tiles, cudaStream_t s) {
  return sdt == kSInt8   ? run_multi<WDT, kSInt8, GDT>(p, tiles, s)
         : sdt == kSBf16 ? run_multi<WDT, kSBf16, GDT>(p, tiles, s)
                         : run_multi<WDT, kSFp32, GDT>(p, tiles, s);
}

}  // namespace

cudaError_t launch_multi(int wdt, int sdt, int gdt, const MultiParams<kMultiLong>& p, uint32_t tiles,
                         cudaStream_t s) {
  if (wdt == kWBf16)
    return gdt == kGBf16 ? run_multi_sdt<kWBf16, kGBf16>(sdt, p, tiles, s)
                         : run_multi_sdt<kWBf16, kGFp32>(sdt, p, tiles, s);
  return gdt == kGBf16 ? run_multi_sdt<kWFp32, kGBf16>(sdt, p, tiles, s)
                       : run_multi_sdt<kWFp32, kGFp32>(sdt, p, tiles, s);
}

}  // namespace forge
