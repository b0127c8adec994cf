// quant.cu -- the prefix cache in 8 bits: writing it (a whole prefix, or a
// committed block) and reading it back.
//
// A page (16 tokens) of K or V of one KV head is 16 x 128 e4m3 codes and one
// fp32 scale, a power of two: x is stored as the e4m3 number nearest to
// x / scale.  Dividing by a power of two is exact, so the code's rounding (half
// a step, 2^-4 of the value; below 2^-6 * scale half of 2^-9 * scale) is the
// only one.  Writing K also writes the page's metadata record over code * scale
// -- the min/max are found on the codes (multiplying by a positive scale keeps
// their order) and scaled once.
//
// All three kernels give one warp to one page of K or V: it reads the page
// once, all of its loads in flight, reduces its largest magnitude in registers,
// and writes codes, scale and record.  The bound is HBM.  A page is the unit that
// shares a scale, so a warp needs no other warp; 4 KB in flight per warp, 16 to 24
// warps per SM, cover the memory's latency.  The kernels are launched behind the
// one ahead of them (programmatic dependent launch), which saves 2 us a call.
// Measured, calls back to back, against the time of the bytes at the copy
// bandwidth (6.45 TB/s), 8 KV heads: reading back a 64K prefix 61.3 us (403 MB:
// 62.5); quantising a 16K prefix with its records 18.1 us (105 MB: 16.3; with the
// elements as floats in place of packed bf16 pairs 6 us more; with 4 blocks per SM
// forced, which spills, a tenth more); appending a block of 16 to 64K 3.9 us,
// which is a launch and two dependent reads: scale and code, then the store.
#include "e4m3.cuh"
#include "losa_common.cuh"

namespace losa {
namespace {

constexpr int kQWarps = 8;
constexpr int kChunk = 8;  // channels per lane: half-warp h of a load takes tokens 2i + h

// Eight elements from element idx on, as floats.
template <int DT>
__device__ __forceinline__ void ld8(const void* base, size_t idx, float (&x)[8]) {
  if (DT == LOSA_BF16) {
    const uint4 r = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(base) + idx));
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  } else {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + idx);
    const float4 a = __ldg(p), b = __ldg(p + 1);
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
    x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  }
}

// Encode one page held in registers -- lane (h = lane / 16, c = lane % 16)
// has channels 8c .. 8c + 7 of tokens 2i + h in x[i], tokens >= n not used --
// and return the scale's exponent; codes[i] are the eight codes of x[i].
__device__ __forceinline__ int encode_page(const float (&x)[8][8], int n, uint2 (&codes)[8]) {
  const int h = (threadIdx.x & 31) >> 4;
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (2 * i + h < n) amax = fmaxf(amax, fabsf(x[i][j]));  // (fmaxf drops a NaN)
  // non-negative floats are ordered like their bits
  amax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(amax)));
  const int e = page_scale_exp(amax);
  const float inv = exp2_int(-e);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    codes[i].x = e4m3x4(x[i][0] * inv, x[i][1] * inv, x[i][2] * inv, x[i][3] * inv);
    codes[i].y = e4m3x4(x[i][4] * inv, x[i][5] * inv, x[i][6] * inv, x[i][7] * inv);
  }
  return e;
}

// The metadata record and norms of page p of group sg: lane (h = lane / 16,
// c = lane % 16) has channels 8c .. of kmin (h = 0) or kmax (h = 1).
template <int DT>
__device__ __forceinline__ void store_record(const float (&v)[8], void* meta, int sg, int p,
                                             const Dims& d) {
  const int lane = threadIdx.x & 31, h = lane >> 4, c = lane & 15;
  // this half's norm, every operation rounded up
  float sum = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) sum = __fmaf_ru(v[j], v[j], sum);
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) sum = __fadd_ru(sum, __shfl_xor_sync(0xffffffffu, sum, o));
  if (c == 0) {
    float* nrm = reinterpret_cast<float*>(static_cast<char*>(meta) + meta_norm_offset(d));
    nrm[(static_cast<size_t>(sg) * meta_norm_stride(d) + p) * 2 + h] = __fsqrt_ru(sum);
  }
  char* rec = static_cast<char*>(meta) + (static_cast<size_t>(sg) * d.Pc + p) * (2 * kD * d.esz);
  if (DT == LOSA_BF16) {
    // four significant bits and an exponent >= -109: exact in bf16
    uint4 w;
    w.x = (__float_as_uint(v[0]) >> 16) | (__float_as_uint(v[1]) & 0xffff0000u);
    w.y = (__float_as_uint(v[2]) >> 16) | (__float_as_uint(v[3]) & 0xffff0000u);
    w.z = (__float_as_uint(v[4]) >> 16) | (__float_as_uint(v[5]) & 0xffff0000u);
    w.w = (__float_as_uint(v[6]) >> 16) | (__float_as_uint(v[7]) & 0xffff0000u);
    *reinterpret_cast<uint4*>(rec + meta_swz(h * 2u * kD + 16u * c, p)) = w;
  } else {
    *reinterpret_cast<float4*>(rec + meta_swz(h * 4u * kD + 32u * c, p)) =
        make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4*>(rec + meta_swz(h * 4u * kD + 32u * c + 16u, p)) =
        make_float4(v[4], v[5], v[6], v[7]);
  }
}

// The same from the page's codes (laid out as in encode_page) and its scale 2^e.
template <int DT>
__device__ __forceinline__ void code_record(const uint2 (&codes)[8], int n, int e, void* meta,
                                            int sg, int p, const Dims& d) {
  const int lane = threadIdx.x & 31, h = lane >> 4;
  // min/max of the codes as fp16 pairs (exact); a half-warp without a token
  // (n = 1) starts from the other one's
  uint32_t lo[4], hi[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    lo[q] = 0x7c007c00u;  // +inf
    hi[q] = 0xfc00fc00u;  // -inf
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (2 * i + h < n) {
      uint32_t f[4];
      e4m3x4_to_f16x2(codes[i].x, f[0], f[1]);
      e4m3x4_to_f16x2(codes[i].y, f[2], f[3]);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        lo[q] = f16x2_min(lo[q], f[q]);
        hi[q] = f16x2_max(hi[q], f[q]);
      }
    }
  }
  // both half-warps get the page's values: half 0 stores kmin, half 1 kmax
  float v[8];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    lo[q] = f16x2_min(lo[q], __shfl_xor_sync(0xffffffffu, lo[q], 16));
    hi[q] = f16x2_max(hi[q], __shfl_xor_sync(0xffffffffu, hi[q], 16));
    const float2 f = f16x2_to_f32(h ? hi[q] : lo[q]);
    const float s = exp2_int(e);
    v[2 * q] = f.x * s;
    v[2 * q + 1] = f.y * s;
  }
  store_record<DT>(v, meta, sg, p, d);
}

// ---- whole pages: the elements stay in their own type until they are encoded
__device__ __forceinline__ uint32_t bf2_min(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("min.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t bf2_max(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// The eight elements of one token that a lane holds.
template <int DT>
struct Row8;
template <>
struct Row8<LOSA_BF16> {
  uint4 w;
  __device__ __forceinline__ void load(const void* base, size_t idx) {
    w = __ldcs(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(base) + idx));
  }
  __device__ __forceinline__ void floats(float (&x)[8]) const {
    const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(v[i] << 16);
      x[2 * i + 1] = __uint_as_float(v[i] & 0xffff0000u);
    }
  }
  __device__ __forceinline__ void minmax(Row8& lo, Row8& hi) const {
    lo.w = make_uint4(bf2_min(lo.w.x, w.x), bf2_min(lo.w.y, w.y), bf2_min(lo.w.z, w.z), bf2_min(lo.w.w, w.w));
    hi.w = make_uint4(bf2_max(hi.w.x, w.x), bf2_max(hi.w.y, w.y), bf2_max(hi.w.z, w.z), bf2_max(hi.w.w, w.w));
  }
  __device__ __forceinline__ void absmax(Row8& m) const {
    constexpr uint32_t k = 0x7fff7fffu;
    m.w = make_uint4(bf2_max(m.w.x, w.x & k), bf2_max(m.w.y, w.y & k), bf2_max(m.w.z, w.z & k),
                     bf2_max(m.w.w, w.w & k));
  }
  __device__ __forceinline__ Row8 other_half() const {
    Row8 r;
    r.w = make_uint4(__shfl_xor_sync(0xffffffffu, w.x, 16), __shfl_xor_sync(0xffffffffu, w.y, 16),
                     __shfl_xor_sync(0xffffffffu, w.z, 16), __shfl_xor_sync(0xffffffffu, w.w, 16));
    return r;
  }
};
template <>
struct Row8<LOSA_F32> {
  float v[8];
  __device__ __forceinline__ void load(const void* base, size_t idx) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + idx);
    const float4 a = __ldcs(p), b = __ldcs(p + 1);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
  __device__ __forceinline__ void floats(float (&x)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = v[i];
  }
  __device__ __forceinline__ void minmax(Row8& lo, Row8& hi) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      lo.v[i] = fminf(lo.v[i], v[i]);
      hi.v[i] = fmaxf(hi.v[i], v[i]);
    }
  }
  __device__ __forceinline__ void absmax(Row8& m) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) m.v[i] = fmaxf(m.v[i], fabsf(v[i]));
  }
  __device__ __forceinline__ Row8 other_half() const {
    Row8 r;
#pragma unroll
    for (int i = 0; i < 8; ++i) r.v[i] = __shfl_xor_sync(0xffffffffu, v[i], 16);
    return r;
  }
};

// Rounding to a code keeps the order, so the codes' min and max over a page are
// the codes of the elements' min and max: K needs no second look at its codes.
template <int DT>
__global__ void __launch_bounds__(kQWarps * 32)
    quantize_kernel(const void* __restrict__ K, const void* __restrict__ V,
                    uint8_t* __restrict__ k8, uint8_t* __restrict__ v8,
                    float* __restrict__ ks, float* __restrict__ vs, void* __restrict__ meta,
                    Dims d) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int sg = blockIdx.y;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, h = lane >> 4, c = lane & 15;
  const int L = seq_len(d, sg / d.Hkv);
  // neighbouring warps take the K and the V of one page
  const int p = blockIdx.x * (kQWarps / 2) + (warp >> 1);
  if (p * kPS >= L) return;
  const bool isk = (warp & 1) == 0;
  const int n = min(kPS, L - p * kPS);
  const size_t e0 = (static_cast<size_t>(sg) * d.Lc + p * kPS) * kD + kChunk * c;
  const void* src = isk ? K : V;
  Row8<DT> x[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)  // (a token past the end: the page's first one again)
    x[i].load(src, e0 + static_cast<size_t>(2 * i + h < n ? 2 * i + h : 0) * kD);
  const bool rec = isk && meta;
  Row8<DT> lo = x[0], hi = x[0];
  float amax = 0.f;
  {
    Row8<DT> m;
    if (rec) {
#pragma unroll
      for (int i = 1; i < 8; ++i) x[i].minmax(lo, hi);
      const Row8<DT> a = lo.other_half(), b = hi.other_half();
      a.minmax(lo, hi);
      b.minmax(lo, hi);
    }
    float f[8];
    if (rec) {
      lo.floats(f);
#pragma unroll
      for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(f[j]));  // (fmaxf drops a NaN)
      hi.floats(f);
    } else {
      m = x[0];
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i].absmax(m);
      m.floats(f);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(f[j]));
  }
  // non-negative floats are ordered like their bits
  amax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(amax)));
  const int e = page_scale_exp(amax);
  const float inv = exp2_int(-e);
  uint8_t* dst = isk ? k8 : v8;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float f[8];
    x[i].floats(f);
    uint2 w;
    w.x = e4m3x4(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv);
    w.y = e4m3x4(f[4] * inv, f[5] * inv, f[6] * inv, f[7] * inv);
    if (2 * i + h < n) *reinterpret_cast<uint2*>(dst + e0 + (2 * i + h) * kD) = w;
  }
  if (lane == 0) (isk ? ks : vs)[static_cast<size_t>(sg) * d.Pc + p] = exp2_int(e);
  if (rec) {
    float f[8], v[8];
    if (h) hi.floats(f);
    else lo.floats(f);
    const float4 a = e4m3x4_to_f32(e4m3x4(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv));
    const float4 b = e4m3x4_to_f32(e4m3x4(f[4] * inv, f[5] * inv, f[6] * inv, f[7] * inv));
    const float s = exp2_int(e);
    v[0] = a.x * s, v[1] = a.y * s, v[2] = a.z * s, v[3] = a.w * s;
    v[4] = b.x * s, v[5] = b.y * s, v[6] = b.z * s, v[7] = b.w * s;
    store_record<DT>(v, meta, sg, p, d);
  }
}

// One warp per touched page of K or V (pages L/ps .. (L+B-1)/ps): the page's
// older tokens are read back (code * scale), its new ones come from the block;
// every load is done before the warp stores, and no other warp touches the
// page.
template <int DT>
__global__ void __launch_bounds__(kQWarps * 32)
    append_quant_kernel(const void* __restrict__ kb, const void* __restrict__ vb, uint8_t* k8,
                        uint8_t* v8, float* ks, float* vs, void* __restrict__ meta, Dims d) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int sg = blockIdx.y;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, h = lane >> 4, c = lane & 15;
  const int L = seq_len(d, sg / d.Hkv);
  const int i0 = blockIdx.x * (kQWarps / 2) + (warp >> 1);
  const int p = L / kPS + i0;
  const int L1 = L + d.B;
  if (p * kPS >= L1) return;
  const bool isk = (warp & 1) == 0;
  const int n = min(kPS, L1 - p * kPS);
  const int nold = max(0, L - p * kPS);  // (only the first page holds older tokens)
  const size_t e0 = (static_cast<size_t>(sg) * d.Lc + p * kPS) * kD + kChunk * c;
  uint8_t* dst = isk ? k8 : v8;
  float* sp = (isk ? ks : vs) + static_cast<size_t>(sg) * d.Pc + p;
  const void* src = isk ? kb : vb;
  const float old = nold > 0 ? *sp : 0.f;
  float x[8][8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int t = 2 * i + h;
    if (t < nold) {
      const uint2 w = *reinterpret_cast<const uint2*>(dst + e0 + t * kD);
      const float4 a = e4m3x4_to_f32(w.x), b = e4m3x4_to_f32(w.y);
      x[i][0] = a.x * old, x[i][1] = a.y * old, x[i][2] = a.z * old, x[i][3] = a.w * old;
      x[i][4] = b.x * old, x[i][5] = b.y * old, x[i][6] = b.z * old, x[i][7] = b.w * old;
    } else {
      const int j = min(max(p * kPS + t - L, 0), d.B - 1);
      ld8<DT>(src, (static_cast<size_t>(sg) * d.B + j) * kD + kChunk * c, x[i]);
    }
  }
  uint2 codes[8];
  const int e = encode_page(x, n, codes);
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (2 * i + h < n) *reinterpret_cast<uint2*>(dst + e0 + (2 * i + h) * kD) = codes[i];
  if (lane == 0) *sp = exp2_int(e);
  if (isk && meta) code_record<DT>(codes, n, e, meta, sg, p, d);
}

template <int DT>
__global__ void __launch_bounds__(kQWarps * 32)
    dequantize_kernel(const uint8_t* __restrict__ k8, const uint8_t* __restrict__ v8,
                      const float* __restrict__ ks, const float* __restrict__ vs,
                      void* __restrict__ K, void* __restrict__ V, Dims d) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int sg = blockIdx.y;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, h = lane >> 4, c = lane & 15;
  const int L = seq_len(d, sg / d.Hkv);
  const int p = blockIdx.x * (kQWarps / 2) + (warp >> 1);
  if (p * kPS >= L) return;
  const bool isk = (warp & 1) == 0;
  const int n = min(kPS, L - p * kPS);
  const size_t e0 = (static_cast<size_t>(sg) * d.Lc + p * kPS) * kD + kChunk * c;
  const uint8_t* src = isk ? k8 : v8;
  const float s = (isk ? ks : vs)[static_cast<size_t>(sg) * d.Pc + p];
  uint2 w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    w[i] = __ldg(reinterpret_cast<const uint2*>(src + e0 + (2 * i + h < n ? 2 * i + h : 0) * kD));
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (2 * i + h >= n) continue;
    const float4 a = e4m3x4_to_f32(w[i].x), b = e4m3x4_to_f32(w[i].y);
    const size_t e = e0 + (2 * i + h) * kD;
    if (DT == LOSA_BF16) {
      __nv_bfloat162 r[4] = {__floats2bfloat162_rn(a.x * s, a.y * s), __floats2bfloat162_rn(a.z * s, a.w * s),
                             __floats2bfloat162_rn(b.x * s, b.y * s), __floats2bfloat162_rn(b.z * s, b.w * s)};
      *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(isk ? K : V) + e) =
          *reinterpret_cast<const uint4*>(r);
    } else {
      float4* o = reinterpret_cast<float4*>(static_cast<float*>(isk ? K : V) + e);
      o[0] = make_float4(a.x * s, a.y * s, a.z * s, a.w * s);
      o[1] = make_float4(b.x * s, b.y * s, b.z * s, b.w * s);
    }
  }
}

// The regions of a quantised cache: codes, then scales.
struct QuantSizes {
  size_t code, scale;
};
QuantSizes quant_sizes(const Dims& d) {
  const size_t SG = static_cast<size_t>(d.S) * d.Hkv;
  return {SG * d.Lc * kD, SG * d.Pc * sizeof(float)};
}

}  // namespace
}  // namespace losa

extern "C" int losa_quantize_prefix(const losa_shape* shape, const void* k_prefix,
                                    const void* v_prefix, void* k8, void* v8, float* k_scale,
                                    float* v_scale, void* page_meta, void* stream) {
  using namespace losa;
  Dims d;
  const int rc = make_dims(shape, LOSA_WS_DENSE, &d);
  if (rc != LOSA_OK) return rc;
  if (bad_ptr(k_prefix) || bad_ptr(v_prefix) || bad_ptr(k8) || bad_ptr(v8) || bad_scale_ptr(k_scale) ||
      bad_scale_ptr(v_scale) || bad_opt_ptr(page_meta))
    return LOSA_ERR_INVALID_ARG;
  const QuantSizes q = quant_sizes(d);
  const size_t pb = q.code * d.esz;
  const Region reg[] = {{k_prefix, pb, false}, {v_prefix, pb, false}, {k8, q.code, true},
                        {v8, q.code, true},    {k_scale, q.scale, true}, {v_scale, q.scale, true},
                        {page_meta, losa_page_meta_size(shape), true}};
  if (any_write_alias(reg, static_cast<int>(sizeof(reg) / sizeof(reg[0]))))
    return LOSA_ERR_INVALID_ARG;
  const dim3 grid((d.P + kQWarps / 2 - 1) / (kQWarps / 2), d.S * d.Hkv);
  if (d.S * static_cast<long long>(d.Hkv) > 65535) return LOSA_ERR_UNSUPPORTED;
  auto* f = d.dtype == LOSA_BF16 ? quantize_kernel<LOSA_BF16> : quantize_kernel<LOSA_F32>;
  return launch_behind(f, grid, kQWarps * 32, 0, static_cast<cudaStream_t>(stream),
                       k_prefix, v_prefix, static_cast<uint8_t*>(k8), static_cast<uint8_t*>(v8),
                       k_scale, v_scale, page_meta, d);
}

extern "C" int losa_append_block_quant(const losa_shape* shape, const void* k_blk,
                                       const void* v_blk, void* k8, void* v8, float* k_scale,
                                       float* v_scale, void* page_meta, void* stream) {
  using namespace losa;
  Dims d;
  const int rc = make_dims(shape, LOSA_WS_DENSE, &d);
  if (rc != LOSA_OK) return rc;
  if (bad_ptr(k_blk) || bad_ptr(v_blk) || bad_ptr(k8) || bad_ptr(v8) || bad_scale_ptr(k_scale) ||
      bad_scale_ptr(v_scale) || bad_opt_ptr(page_meta))
    return LOSA_ERR_INVALID_ARG;
  if (static_cast<long long>(d.L) + d.B > d.Lc) return LOSA_ERR_INVALID_ARG;  // no room
  const QuantSizes q = quant_sizes(d);
  const size_t bb = static_cast<size_t>(d.S) * d.Hkv * d.B * kD * d.esz;
  const Region reg[] = {{k_blk, bb, false},   {v_blk, bb, false},        {k8, q.code, true},
                        {v8, q.code, true},   {k_scale, q.scale, true},  {v_scale, q.scale, true},
                        {page_meta, losa_page_meta_size(shape), true}};
  if (any_write_alias(reg, static_cast<int>(sizeof(reg) / sizeof(reg[0]))))
    return LOSA_ERR_INVALID_ARG;
  if (d.S * static_cast<long long>(d.Hkv) > 65535) return LOSA_ERR_UNSUPPORTED;
  // pages touched: (L+B-1)/ps - L/ps + 1 <= (B-1)/ps + 2, whatever L is
  const int np = (d.B - 1) / kPS + 2;
  const dim3 grid((np + kQWarps / 2 - 1) / (kQWarps / 2), d.S * d.Hkv);
  auto* f = d.dtype == LOSA_BF16 ? append_quant_kernel<LOSA_BF16> : append_quant_kernel<LOSA_F32>;
  return launch_behind(f, grid, kQWarps * 32, 0, static_cast<cudaStream_t>(stream),
                       k_blk, v_blk, static_cast<uint8_t*>(k8), static_cast<uint8_t*>(v8),
                       k_scale, v_scale, page_meta, d);
}

extern "C" int losa_dequantize_prefix(const losa_shape* shape, const void* k8, const void* v8,
                                      const float* k_scale, const float* v_scale, void* k_prefix,
                                      void* v_prefix, void* stream) {
  using namespace losa;
  Dims d;
  const int rc = make_dims(shape, LOSA_WS_DENSE, &d);
  if (rc != LOSA_OK) return rc;
  if (bad_ptr(k8) || bad_ptr(v8) || bad_scale_ptr(k_scale) || bad_scale_ptr(v_scale) || bad_ptr(k_prefix) ||
      bad_ptr(v_prefix))
    return LOSA_ERR_INVALID_ARG;
  const QuantSizes q = quant_sizes(d);
  const size_t pb = q.code * d.esz;
  const Region reg[] = {{k_prefix, pb, true},    {v_prefix, pb, true},     {k8, q.code, false},
                        {v8, q.code, false},     {k_scale, q.scale, false}, {v_scale, q.scale, false}};
  if (any_write_alias(reg, static_cast<int>(sizeof(reg) / sizeof(reg[0]))))
    return LOSA_ERR_INVALID_ARG;
  const dim3 grid((d.P + kQWarps / 2 - 1) / (kQWarps / 2), d.S * d.Hkv);
  if (d.S * static_cast<long long>(d.Hkv) > 65535) return LOSA_ERR_UNSUPPORTED;
  auto* f = d.dtype == LOSA_BF16 ? dequantize_kernel<LOSA_BF16> : dequantize_kernel<LOSA_F32>;
  return launch_behind(f, grid, kQWarps * 32, 0, static_cast<cudaStream_t>(stream),
                       static_cast<const uint8_t*>(k8), static_cast<const uint8_t*>(v8), k_scale,
                       v_scale, k_prefix, v_prefix, d);
}
