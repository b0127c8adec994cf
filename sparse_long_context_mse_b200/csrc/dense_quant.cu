// dense_quant.cu -- the dense pass over a prefix cache held in 8 bits.
//
// s_j = scale * ks(page j) * (q . k8_j);  o = sum_j e^(s_j - m) vs(page j) v8_j
// / sum_j e^(s_j - m): the page scales are factors of a key's score and of its
// value.  Flash-decode layout as in dense.cu: one CTA streams a range of pages
// for all G*B query rows of a KV head and writes an online-softmax partial per
// row; the finish kernel merges them.
#include "e4m3.cuh"
#include "losa_common.cuh"

namespace losa {
namespace {

constexpr int kWarpsQ = 8;
constexpr int kRowsQ = 8;  // query rows per warp

// One page of codes into shared memory as fp32 values, rows >= ntok zero.
__device__ __forceinline__ void load_page_e4m3(const uint8_t* src, float s, int ntok, float* dst) {
  const int j = threadIdx.x >> 4, c = (threadIdx.x & 15) * 8;  // 256 threads: 16 rows x 16 chunks
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
  if (j < ntok) {
    const uint2 w = *reinterpret_cast<const uint2*>(src + j * kD + c);
    a = e4m3x4_to_f32(w.x);
    b = e4m3x4_to_f32(w.y);
  }
  float4* o = reinterpret_cast<float4*>(dst + j * kD + c);
  o[0] = make_float4(a.x * s, a.y * s, a.z * s, a.w * s);
  o[1] = make_float4(b.x * s, b.y * s, b.z * s, b.w * s);
}

__global__ void __launch_bounds__(kWarpsQ * 32)
    dense_quant_partial_kernel(const void* __restrict__ Q, const uint8_t* __restrict__ K,
                               const uint8_t* __restrict__ V, const float* __restrict__ ks,
                               const float* __restrict__ vs, float* __restrict__ part,
                               int* __restrict__ status, Dims d) {
  __shared__ __align__(16) float Ks[kPS * kD];
  __shared__ __align__(16) float Vs[kPS * kD];
  __shared__ float Ps[kWarpsQ][kPS];
  const int sg = blockIdx.y, split = blockIdx.x;
  const int s = sg / d.Hkv, g = sg % d.Hkv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rows = d.G * d.B;
  const int L = seq_len(d, s);
  const int p0 = split * d.split_pages;
  const int p1 = min((L + kPS - 1) / kPS, p0 + d.split_pages);
  if (split == 0 && threadIdx.x == 0 && seq_len_bad(d, s)) atomicCAS(status, 0, LOSA_ERR_DEVICE_BOUNDS);
  for (int rbase = 0; rbase < rows; rbase += kWarpsQ * kRowsQ) {
    float4 q[kRowsQ], acc[kRowsQ];
    float m[kRowsQ], l[kRowsQ];
#pragma unroll
    for (int i = 0; i < kRowsQ; ++i) {
      const int r = rbase + warp * kRowsQ + i;
      const int rr = r < rows ? r : 0;
      const int h = g * d.G + rr / d.B, t = rr % d.B;
      q[i] = ld4(Q, ((static_cast<size_t>(s) * d.Hq + h) * d.B + t) * kD + 4 * lane, d.dtype);
      acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      m[i] = -INFINITY;
      l[i] = 0.f;
    }
    for (int p = p0; p < p1; ++p) {
      const int ntok = min(kPS, L - p * kPS);
      const size_t off = (static_cast<size_t>(sg) * d.Lc + static_cast<size_t>(p) * kPS) * kD;
      const size_t sp = static_cast<size_t>(sg) * d.Pc + p;
      __syncthreads();
      load_page_e4m3(K + off, ks[sp], ntok, Ks);
      load_page_e4m3(V + off, fmaxf(vs[sp], kMinScale), ntok, Vs);
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kRowsQ; ++i)
        if (rbase + warp * kRowsQ + i < rows)
          attend_page_row(q[i], Ks, Vs, ntok, d.scale_log2, m[i], l[i], acc[i], Ps[warp]);
    }
#pragma unroll
    for (int i = 0; i < kRowsQ; ++i) {
      const int r = rbase + warp * kRowsQ + i;
      if (r >= rows) continue;
      float* dst = part + ((static_cast<size_t>(sg) * d.nsplit + split) * rows + r) * kPartStride;
      if (lane == 0) {
        dst[0] = m[i];
        dst[1] = l[i];
      }
      *reinterpret_cast<float4*>(dst + 4 + 4 * lane) = acc[i];
    }
  }
}

}  // namespace
}  // namespace losa

extern "C" int losa_dense_prefix_quant(const losa_shape* shape, const void* q, const void* k8,
                                       const void* v8, const float* k_scale, const float* v_scale,
                                       const void* k_blk, const void* v_blk, float* o_p,
                                       float* l_p, float* out, float* out_lse, void* workspace,
                                       size_t ws_bytes, void* stream) {
  using namespace losa;
  Dims d;
  int rc = make_dims(shape, LOSA_WS_DENSE_QUANT, &d);
  if (rc != LOSA_OK) return rc;
  if (bad_ptr(q) || bad_ptr(k8) || bad_ptr(v8) || bad_scale_ptr(k_scale) || bad_scale_ptr(v_scale) ||
      bad_ptr(k_blk) || bad_ptr(v_blk) || bad_ptr(o_p) || bad_ptr(l_p) || bad_ptr(out) ||
      bad_opt_ptr(out_lse) || !workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u))
    return LOSA_ERR_INVALID_ARG;
  if (ws_bytes < d.total) return LOSA_ERR_INVALID_ARG;
  const size_t rows = static_cast<size_t>(d.S) * d.Hq * d.B;
  const size_t SG = static_cast<size_t>(d.S) * d.Hkv;
  const size_t qb = rows * kD * d.esz, ob = rows * kD * sizeof(float), lb = rows * sizeof(float);
  const size_t cb = SG * d.Lc * kD, sb = SG * d.Pc * sizeof(float), kbb = SG * d.B * kD * d.esz;
  const Region reg[] = {{q, qb, false},       {k8, cb, false},       {v8, cb, false},
                        {k_scale, sb, false}, {v_scale, sb, false},  {k_blk, kbb, false},
                        {v_blk, kbb, false},  {o_p, ob, true},       {l_p, lb, true},
                        {out, ob, true},      {out_lse, lb, true},   {workspace, d.total, true}};
  if (any_write_alias(reg, static_cast<int>(sizeof(reg) / sizeof(reg[0]))))
    return LOSA_ERR_INVALID_ARG;
  if (SG > 65535) return LOSA_ERR_UNSUPPORTED;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  float* part = reinterpret_cast<float*>(static_cast<char*>(workspace) + d.off_part);
  int* status = reinterpret_cast<int*>(static_cast<char*>(workspace) + d.off_status);
  dense_quant_partial_kernel<<<dim3(d.nsplit, static_cast<unsigned>(SG)), kWarpsQ * 32, 0, st>>>(
      q, static_cast<const uint8_t*>(k8), static_cast<const uint8_t*>(v8), k_scale, v_scale, part,
      status, d);
  rc = launch_dense_finish(d, q, k_blk, v_blk, part, o_p, l_p, out, out_lse, st);
  if (rc != LOSA_OK) return rc;
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? LOSA_OK : record_cuda_error(e);
}
