// dense_quant.cu -- the dense pass over a prefix cache held in 8 bits.
//
// The page scales are factors of a key's score and of its value.  In base 2, with
// x_j = scale * ks(page j) * (q . k8_j) * log2(e), a reference m per row and a power
// of two 2^E, 2^40 below the largest V scale, the kernel accumulates
//
//   p_j = 2^(x_j - m),   l = sum_j p_j,   W_j = p_j vs(page j) 2^-E,
//   O = sum_j W_j v8_j,   o = 2^E O / l,
//
// E is that of the first tile of a KV head's keys and moves, as a reference does, when
// a tile's largest scale passes 2^(E + 40 + 32): nothing overflows, whatever the size of
// the V scales, and a key keeps all of its bits while p is a normal number (2^-126) and
// p vs is not below 2^-140 of the largest V scale.
//
// Its floor is HBM: 256 bytes per key and KV head, read once.  The work is laid
// out so that little on the chip takes longer:
//
// * Keys are the rows of both products (M = 128, one tile), the G*B query rows
//   are the columns (N = 16, 32 or 64; 128 rows take two CTAs that read the same
//   keys at the same time, the second time from L2): few query rows cost little.
// * S^T = K8 Q^T runs on the codes as TMA brought them (kind::f8f6f4, e4m3 times
//   e4m3): nothing converts K.  Q enters as a sum of 8-bit parts, each the
//   rounding of what the parts before it left, rows scaled by a power of two to a
//   maximum in [128, 256).  A bf16 number has 8 significant bits: an e4m3 part
//   holds 4, and what rounding to nearest leaves, -8 .. 8 units of the last place,
//   has 3 at most, which is an e5m2 number.  So the two are exact down to 2^-13 of
//   the row's maximum, and within 2^-21 of it below (an e4m3 second part, with its
//   smaller range: 2^-17, and twice the results' error).  fp32 takes six e4m3
//   parts, the last three 2^12 times larger in an accumulator of their own, within
//   2^-29 of the row's maximum.
// * O^T = V8^T W: W as the sum of three bf16 numbers, its top, middle and low 8
//   bits: all 24 of an fp32 number, at any size an fp32 number can have.  What holds
//   a row's weight need not be what its output is made of (a page or a token of
//   zeros, values far smaller than another page's), so a weight keeps its own
//   relative accuracy, however far it lies below the reference.  (Two fp16 parts
//   are cheaper -- 64 rows, 64K prefix 43 us in place of 47 -- and have 22 bits, but
//   only of weights within 2^-13 of the largest; below 2^-36 they are zero.)  V8 has
//   to be bf16 too.  Four warps transpose V codes out of shared memory (ldmatrix,
//   bytes), widen them (exact) and store them as the A operand in TMEM, which costs
//   1/8 of the shared-memory traffic of a 16-bit tile there; W goes through shared
//   memory as the MN-major B.
// * A softmax thread owns one key (TMEM lane) and 8 or 16 of the query columns:
//   the page scales are constants of the thread, l is a sum in registers across tiles
//   (joined over the lanes at the end), and no tile needs a maximum over the
//   lanes: the reference moves only when some p would pass 2^4, which one
//   barrier with a vote finds out.
// * The tensor core's accumulator truncates (up to 2^-24 of it on each of the 24
//   steps of a tile, all in one direction: 1.4e-5 after 800 of them, measured),
//   so O stays in it for one tile only and is summed in registers.
// * All SMs get the same number of tiles, whatever the lengths and the number of
//   KV heads (the line of tiles, losa_common.cuh).
//
// Measured, calls back to back (with the finish kernel; the floor at the copy
// bandwidth of 6.45 TB/s): 8 KV heads, 64K prefix, 134 MB, floor 21 us: 16 rows
// per KV head 31.1 us, 32 rows 35.4, 64 rows 47.0; fp32 38.2, 41.1, 54.4.  With 16
// rows it is bound by the loads (what is left of it with the softmax taken out takes
// 28 us: 23 for the bytes, and a prologue and an end that no tile overlaps).  With 64
// rows a tile's 2300 cycles go to the softmax warps and to widening V: 8192 weights,
// each scaled, voted on, raised to a power of two and split in three, and 16384
// codes, some 6300 warp instructions at 62 % of the issue slots, the tensor core at
// 40 %.  Eight sequences of 32K and 128 rows (two CTAs each range), floor 85 us: 296
// us, the same.  In loops of more than a few milliseconds the 64-row passes draw the
// card's 1000 W and the clock falls from 1.92 to 1.65 GHz: 52 and 346 us.
#include "device_once.h"
#include "e4m3.cuh"
#include "losa_common.cuh"
#include "ptx.cuh"
#include "umma.cuh"

namespace losa {
namespace {

// Softmax warp groups first (2, or 4 for 64 columns), then four warps that widen
// V, then one that loads, one that issues MMAs, one that prepares the tiles'
// scales and one that has nothing to do.
constexpr int kTileBytes = kLineKeys * kD;  // one K or V tile of codes: 16 KB
constexpr int kVCols = kLineKeys / 2;       // TMEM columns of a V^T tile (bf16 pairs)
// A row's reference is its largest score when it is set, and stays until a weight would
// pass 2^4; E likewise.  So a key adds at most 2^(4 + 33 + 40 + 9) to O, and 2^30 keys
// (more than the card has memory for) stay below 2^116; a weight of 2^-100 still has
// its third part above bf16's smallest number.
constexpr float kRefMove = 4.f;
constexpr int kScaleMove = 32, kScaleUp = 40;
constexpr float kPartScale = 4096.f;        // fp32: parts 4-6 are this much larger

typedef unsigned long long u64;

// Pairs of fp32 numbers in one 64-bit register pair.
__device__ __forceinline__ u64 pk(float a, float b) {
  u64 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 up(u64 a) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a));
  return r;
}
__device__ __forceinline__ u64 mul2(u64 a, u64 b) {
  u64 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ u64 add2(u64 a, u64 b) {
  u64 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ u64 fma2(u64 a, u64 b, u64 c) {
  u64 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// NR: query columns (MMA N); NQ: 8-bit parts of a query row (2: bf16, 6: fp32).
template <int NR, int NQ>
struct QPlan {
  // A tile is a chain of dependent waits and instructions for a softmax warp, and
  // the longer the more columns it has, so the columns are spread over as many
  // warps as the registers allow: 16 columns per thread at most, 8 with 32 columns
  // of bf16 queries (64K prefix, 8 KV heads: 35.7 us a pass with four warp groups,
  // 37.2 with two; fp32, with a second score accumulator to read, 42.9 and 41.8).
  // Measured while weights had two parts: 64 columns in four warp groups 51 us, in two
  // 59; one CTA with 128 columns in place of two with 64 346 us for 8 x 32K, against
  // 293.
  static constexpr int nwg = NR > 32 || (NR == 32 && NQ == 2) ? 4 : 2;  // softmax warp groups
  static constexpr int soft = nwg * 128;                 // .. threads
  static constexpr int threads = soft + 256;
  // the softmax warps take registers over from the others
  static constexpr int regs = nwg == 4 ? 80 : 128;       // at launch
  static constexpr int soft_regs = nwg == 4 ? 96 : 192, other_regs = nwg == 4 ? 48 : 64;
  static_assert(soft * soft_regs + 256 * other_regs <= threads * regs, "register split");
  static constexpr int cw = NR / nwg;                    // columns per softmax warp group
  static constexpr int na = NQ > 3 ? 2 : 1;              // score accumulators
  static constexpr int atom = kLineKeys * 128;           // 64 bf16 columns of W: 16 KB
  static constexpr int wbytes = 3 * atom;                // the three parts of W
  static constexpr int qbytes = NQ * NR * kD;
  static constexpr int small = 3 * 1024;                    // barriers, row factors, exchange
  static constexpr int room = kB200MaxDynSmem - small - qbytes - 2 * wbytes;
  static constexpr int st = room / (2 * kTileBytes) < 4 ? room / (2 * kTileBytes) : 4;
  static constexpr int nbars = 7 + 4 * st;
  static constexpr int smem = qbytes + 2 * wbytes + 2 * st * kTileBytes + small;
  static constexpr uint32_t tS = 0, tO = 2 * na * NR, tV = tO + 2 * NR, cols = 512;
  static_assert(NR <= 64 && st >= 2 && smem <= kB200MaxDynSmem, "shared memory");
  static_assert(tV + 2 * kVCols <= 512, "TMEM");
  static_assert(nbars * 8 + 8 + 7 * NR * 4 + 2 * 128 + 64 <= small,
                "small area");
};

// What the softmax warps have to know of a tile.
struct __align__(16) TileInfo {
  // a page's score factor and its value scale times 2^-E; and, in every entry, E and
  // the tile's real keys, + 256 if it is the KV head's last in this CTA
  float4 page[kLineKeys / kPS];
};

// A CTA's place on the line of tiles.
struct LinePos {
  int s, g, lt, nt, L;  // sequence, KV head, tile of it, its number of tiles, its keys
  __device__ __forceinline__ void start(const Dims& d) {
    L = seq_len(d, s);
    nt = (L + kLineKeys - 1) / kLineKeys;
  }
  __device__ __forceinline__ void next_head(const Dims& d) {
    lt = 0;
    if (++g < d.Hkv) return;
    g = 0;
    if (++s < d.S) start(d);
  }
  __device__ __forceinline__ void next(const Dims& d) {
    if (++lt == nt) next_head(d);
  }
};

template <int NR, int NQ>
__global__ void __launch_bounds__(QPlan<NR, NQ>::threads, 1)
    dense_quant_kernel(const void* __restrict__ Q, const __grid_constant__ CUtensorMap kmap,
                       const __grid_constant__ CUtensorMap vmap, const float* __restrict__ ks,
                       const float* __restrict__ vs, float* __restrict__ part,
                       int* __restrict__ status, Dims d) {
  using C = QPlan<NR, NQ>;
  constexpr int CW = C::cw, ST = C::st, NA = C::na, NS = C::soft, W0 = NS / 32;
  extern __shared__ __align__(1024) char sm[];
  if (su32(sm) & 1023u) {  // (the swizzled tiles; dynamic shared memory starts at 1 KB)
    if (threadIdx.x == 0) atomicCAS(status, 0, LOSA_ERR_DEVICE_BOUNDS);
    return;
  }
  char* qs = sm;                              // NQ parts of [NR][128 B]
  char* wbuf = qs + C::qbytes;                // [2] W buffers: [3 (parts)][128][128 B]
  char* kring = wbuf + 2 * C::wbytes;         // ST K tiles
  char* vring = kring + ST * kTileBytes;      // ST V tiles
  uint64_t* bars = reinterpret_cast<uint64_t*>(vring + ST * kTileBytes);
  uint64_t* bS = bars;           // [2] S^T and the info of an even / odd tile ready (MMA, scales)
  uint64_t* bO = bars + 2;       // [2] O = V W of an even / odd tile done
  uint64_t* bP = bars + 4;       // [2] W and V^T of an even / odd tile written (softmax and V warps)
  uint64_t* bQ = bars + 6;       // query parts staged (softmax warps)
  uint64_t* bKf = bars + 7;      // [ST] K tile landed
  uint64_t* bKe = bKf + ST;      // [ST] its MMAs done
  uint64_t* bVf = bKe + ST;      // [ST] V tile landed
  uint64_t* bVe = bVf + ST;      // [ST] read (4 warps)
  float* rf = reinterpret_cast<float*>(bars + C::nbars + 1);  // [NR] 2^-c: undoes a row's scaling
  float* nm = rf + NR;           // [NR] minus the row's reference (+inf: none yet)
  float* xch = nm + NR;          // [warp groups][4][columns] warp maxima / sums
  float* alpha = xch + 4 * NR;   // [NR] factors of a moved reference
  TileInfo* info = reinterpret_cast<TileInfo*>(alpha + NR);  // [2]
  int* line = reinterpret_cast<int*>(info + 2);  // tiles of this CTA, then s, g, lt of the first
  uint32_t* tslot = reinterpret_cast<uint32_t*>(line + 4);
  int* s_fail = reinterpret_cast<int*>(tslot + 1);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int rows = d.G * d.B, r0 = blockIdx.y * NR, nrows = min(NR, rows - r0);

  if (tid == 0) {
    for (int i = 0; i < C::nbars; ++i)
      mbar_init(&bars[i], i < 2 ? 2 : i < 4 ? 1 : i < 6 ? W0 + 4 : i == 6 ? W0 : i >= 7 + 3 * ST ? 4 : 1);
    fence_mbar_init();
    *s_fail = 0;
  }
  // launched with programmatic stream serialisation: nothing is read or written
  // before the work queued ahead has completed.  Only then may the finish kernel
  // be scheduled: it reads the queries and the block before its own wait
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (warp == 1) tmem_alloc(tslot, C::cols);
  if (warp == 0) {
    // this CTA's range of the line, and where it starts
    long long before, all;
    line_sums(d, 0, before, all);
    const long long total = all * d.Hkv;
    const int n = line_ctas_used(d, total), b = blockIdx.x;
    const long long x0 = b < n ? line_div(b * total, n) : 0;
    const long long x1 = b < n ? line_div((b + 1) * total, n) : 0;
    int s = 0;
    before = 0;
    if (d.lens) {
      bool found = false;
      for (int s0 = 0; s0 < d.S && !found; s0 += 32) {
        const int i = s0 + lane;
        int incl = i < d.S ? line_tiles(d, i) : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += y;
        }
        const uint32_t past = __ballot_sync(0xffffffffu, (before + incl) * d.Hkv > x0);
        found = past != 0;
        const int at = found ? __ffs(past) - 1 : 31;
        const int upto = __shfl_sync(0xffffffffu, incl, at > 0 ? at - 1 : 0);
        const int last = __shfl_sync(0xffffffffu, incl, 31);
        s = s0 + at;
        before += found ? (at > 0 ? upto : 0) : last;
      }
    } else {
      const long long nt = (d.L + kLineKeys - 1) / kLineKeys;
      s = static_cast<int>(line_div(x0, nt * d.Hkv));
      before = nt * s;
    }
    if (lane == 0) {
      const long long nt = line_tiles(d, s), y = x0 - before * d.Hkv;
      line[0] = static_cast<int>(x1 - x0);
      line[1] = s;
      line[2] = static_cast<int>(line_div(y, nt));
      line[3] = static_cast<int>(y - nt * line[2]);
    }
    if (b == 0 && blockIdx.y == 0)
      for (int i = lane; d.lens && i < d.S; i += 32)
        if (seq_len_bad(d, i)) atomicCAS(status, 0, LOSA_ERR_DEVICE_BOUNDS);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tb = __shfl_sync(0xffffffffu, *tslot, 0);
  const int n = __shfl_sync(0xffffffffu, line[0], 0);  // this CTA's tiles
  LinePos pos;
  pos.s = __shfl_sync(0xffffffffu, line[1], 0);
  pos.g = __shfl_sync(0xffffffffu, line[2], 0);
  pos.lt = __shfl_sync(0xffffffffu, line[3], 0);
  pos.start(d);
  if (warp >= W0) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::other_regs));
    if (warp == W0 + 4 && n > 0) {
      // ---- loads: K and V tiles through rings of ST stages, one thread
      if (lane == 0) {
        prefetch_tmap(&kmap);
        prefetch_tmap(&vmap);
        int it = 0;
        bool ok = true;
#pragma unroll 1
        for (; it < n; ++it) {
          const int st = it % ST, use = it / ST;
          const int row = (pos.s * d.Hkv + pos.g) * d.Lc + pos.lt * kLineKeys;
          if (use > 0) ok = mbar_wait(&bKe[st], (use - 1) & 1);
          if (!ok) break;
          mbar_expect_tx(&bKf[st], kTileBytes);
          tma_load_2d(kring + st * kTileBytes, &kmap, 0, row, &bKf[st]);
          if (use > 0) ok = mbar_wait(&bVe[st], (use - 1) & 1);
          if (!ok) break;
          mbar_expect_tx(&bVf[st], kTileBytes);
          tma_load_2d(vring + st * kTileBytes, &vmap, 0, row, &bVf[st]);
          pos.next(d);
        }
        if (!ok) {
          // the copies in flight land before the CTA's shared memory goes (each
          // stage's last one is its latest phase; tile it's K copy may be out)
          *s_fail = 1;
          for (int j = max(0, it - ST); j < it; ++j) {
            mbar_wait(&bKf[j % ST], (j / ST) & 1);
            mbar_wait(&bVf[j % ST], (j / ST) & 1);
          }
          mbar_wait(&bKf[it % ST], (it / ST) & 1);
        }
      }
    } else if (warp == W0 + 5 && n > 0) {
      // ---- MMAs: the whole warp follows the loop, one elected thread issues
      constexpr uint32_t idS = umma_idesc_e4m3(128, NR);
      constexpr uint32_t idS2 = umma_idesc_e4m3(128, NR, NQ == 2);
      constexpr uint32_t idO = umma_idesc_bf16(128, NR, 1);
      constexpr uint32_t idM = idO | (1u << 14);  // minus B: the middle part is stored negated
      const uint64_t dq = umma_desc(su32(qs), 16, 1024), dk = umma_desc(su32(kring), 16, 1024);
      const uint64_t dw = umma_desc(su32(wbuf), C::atom, 1024);
      const uint32_t q_lo = desc_lo(dq), k_lo = desc_lo(dk), kq_hi = desc_hi(dq);
      const uint32_t w_lo = desc_lo(dw), w_hi = desc_hi(dw);
      int seg = 0;  // query tiles staged so far
      int ks_ = 0, kph = 0;  // K stage and phase of the next S^T
      auto issue_s = [&](int par, bool fresh) {  // the next S^T, into buffer par
        if (fresh) {
          mbar_wait_or(bQ, seg & 1, s_fail);
          ++seg;
        }
        mbar_wait_or(&bKf[ks_], kph, s_fail);
        __syncwarp();
        tc_fence_after();
        const uint32_t kl = k_lo + ((ks_ * kTileBytes) >> 4);
        const uint32_t ts = tb + C::tS + par * (NA * NR);
        const uint32_t me = elect_one();
        // the small parts first: the sum is truncated to its size at every step
#pragma unroll
        for (int a = NA - 1; a >= 0; --a)
#pragma unroll
          for (int p = NQ / NA - 1; p >= 0; --p)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint32_t ql = q_lo + (((a * (NQ / NA) + p) * NR * kD + k * 32) >> 4);
              const uint32_t id = p > 0 ? idS2 : idS;
              if (p < NQ / NA - 1 || k > 0)
                umma_e4m3<true>(me, ts + a * NR, kl + ((k * 32) >> 4), ql, kq_hi, id);
              else
                umma_e4m3<false>(me, ts + a * NR, kl + ((k * 32) >> 4), ql, kq_hi, id);
            }
        umma_commit_if(me, &bS[par]);
        umma_commit_if(me, &bKe[ks_]);
        if (++ks_ == ST) {
          ks_ = 0;
          kph ^= 1;
        }
      };
      issue_s(0, true);
#pragma unroll 1
      for (int it = 0; it < n; ++it) {
        const int par = it & 1;
        pos.next(d);
        const bool more = it + 1 < n, fresh = pos.lt == 0;
        // the next tile's scores run during this tile's softmax, unless they
        // wait for the next KV head's queries, which are staged after it
        if (more && !fresh) issue_s(par ^ 1, false);
        mbar_wait_or(&bP[par], (it >> 1) & 1, s_fail);
        __syncwarp();
        tc_fence_after();
        const uint32_t wl = w_lo + ((par * C::wbytes) >> 4);
        const uint32_t to = tb + C::tO + par * NR, tv = tb + C::tV + par * kVCols;
        const uint32_t me = elect_one();
#pragma unroll
        for (int h = 2; h >= 0; --h)  // (the small parts first)
#pragma unroll
          for (int k = 0; k < kLineKeys / 16; ++k) {
            const uint32_t b = wl + ((h * C::atom + k * 16 * 128) >> 4);
            if (h == 2 && k == 0)
              umma_f16_ta<false>(me, to, tv + k * 8, b, w_hi, idO);
            else
              umma_f16_ta<true>(me, to, tv + k * 8, b, w_hi, h == 1 ? idM : idO);
          }
        umma_commit_if(me, &bO[par]);
        if (more && fresh) issue_s(par ^ 1, true);
      }
    } else if (warp == W0 + 6 && n > 0) {
      // ---- a tile's scales: lane p < 8 its page p's, read a tile ahead
      float k_ = 1.f, v_ = 0.f;
      auto fetch = [&]() {
        const int j = pos.lt * kLineKeys + lane * kPS;
        k_ = 1.f;
        v_ = 0.f;
        if (lane < kLineKeys / kPS && j < pos.L) {
          const size_t i = static_cast<size_t>(pos.s * d.Hkv + pos.g) * d.Pc + (j >> 4);
          k_ = __ldg(ks + i);
          v_ = __ldg(vs + i);
        }
      };
      fetch();
      int E = 0;
#pragma unroll 1
      for (int it = 0; it < n; ++it) {
        const int nv = min(kLineKeys, pos.L - pos.lt * kLineKeys);
        // (non-negative floats are ordered like their bits)
        const uint32_t top = __reduce_max_sync(0xffffffffu, __float_as_uint(fmaxf(v_, 0.f)));
        const int e = max(static_cast<int>(top >> 23) - 127 - kScaleUp, -126);
        if (it == 0 || pos.lt == 0 || e > E + kScaleMove) E = e;
        pos.next(d);
        const bool last = it + 1 == n || pos.lt == 0;
        const float4 w = make_float4(k_ * d.scale_log2, v_ * exp2_int(-E), __int_as_float(E),
                                     __int_as_float(nv + (last ? 256 : 0)));
        if (it + 1 < n) fetch();
        // (the info of two tiles back has been read)
        if (it >= 2) mbar_wait_or(&bP[it & 1], ((it - 2) >> 1) & 1, s_fail);
        if (lane < kLineKeys / kPS) info[it & 1].page[lane] = w;
        __syncwarp();
        if (lane == 0) mbar_arrive(&bS[it & 1]);
      }
    } else if (warp < W0 + 4) {
      // ---- V codes -> bf16, transposed, into TMEM: warp w4 has the channels
      // 32 w4 .. (its TMEM lanes)
      const int w4 = warp & 3;
      const uint32_t lane_off = static_cast<uint32_t>(w4 * 32) << 16;
#pragma unroll 1
      for (int it = 0; it < n; ++it) {
        const int nv = min(kLineKeys, pos.L - pos.lt * kLineKeys);
        mbar_wait_or(&bVf[it % ST], (it / ST) & 1, s_fail);
        const uint32_t vt = su32(vring + (it % ST) * kTileBytes);
        // V^T of this parity is free once O = V W of two tiles back is done
        if (it >= 2) mbar_wait_or(&bO[it & 1], ((it - 2) >> 1) & 1, s_fail);
        __syncwarp();
        tc_fence_after();
#pragma unroll
        for (int dh = 0; dh < 2; ++dh) {
          uint32_t c[16];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int j = i * 16 + (lane & 15);
            ldsm_b8_trans(vt + j * 128 + (((2 * w4 + dh) ^ (j & 7)) << 4), c[2 * i], c[2 * i + 1]);
          }
          if (nv < kLineKeys) {
            // keys past the prefix may hold anything, and 0 times NaN is NaN
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int m = min(max(nv - (i * 16 + 4 * (lane & 3)), 0), 4);
              const uint32_t mask = m == 4 ? 0xffffffffu : (1u << (8 * m)) - 1u;
              c[2 * i] &= mask;
              c[2 * i + 1] &= mask;
            }
          }
#pragma unroll
          for (int kq = 0; kq < 2; ++kq) {
            uint32_t f[16];
#pragma unroll
            for (int i = 0; i < 8; ++i) e4m3x4_to_bf16x2(c[kq * 8 + i], f[2 * i], f[2 * i + 1]);
            tmem_st16x256_x4_raw(tb + C::tV + (it & 1) * kVCols + kq * 32 + lane_off +
                                     (static_cast<uint32_t>(dh * 16) << 16),
                                 f);
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&bVe[it % ST]);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bP[it & 1]);
        pos.next(d);
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::soft_regs));
    // ---- softmax warps: warp w has TMEM lanes 32 (w % 4) .., keys of the S^T
    // tile and channels of O^T; warp group w / 4 has the query columns c0 ..
    const int w4 = warp & 3, wg = warp >> 2, c0 = wg * CW;
    const uint32_t lane_off = static_cast<uint32_t>(w4 * 32) << 16;
    const int key = 32 * w4 + lane;
    float* xg = xch + wg * 4 * CW;
    float* ag = alpha + wg * CW;
    u64 l[CW / 2], o[CW / 2];
    bool fresh = true;
    int E = 0;  // of what o holds
    bool pend1 = false, pend2 = false;  // O of one / two tiles back is still to be read

    // o += O buffer b (one tile's product)
    auto o_addr = [&](int b) { return tb + C::tO + b * NR + c0 + lane_off; };
    auto add_o = [&](const float (&t)[CW]) {
#pragma unroll
      for (int i = 0; i < CW; i += 2) o[i / 2] = add2(o[i / 2], pk(t[i], t[i + 1]));
    };
    auto take_o = [&](int b) {
      float t[CW];
      tmem_ld_async(o_addr(b), t);
      tmem_ld_wait(t);
      add_o(t);
    };
    auto s_addr = [&](int it, int a) {
      return tb + C::tS + (it & 1) * (NA * NR) + a * NR + c0 + lane_off;
    };
    // the scores as exponents of 2: S rf kf, less the reference in one rounding (ref:
    // a score that makes a new reference and the weights of its tile are the rounded
    // product instead, so that the largest weight is 1 however large the scores are)
    auto to_x = [&](int it, u64 kf2, bool ref, const float (&a)[CW], u64 (&y)[CW / 2]) {
#pragma unroll
      for (int i = 0; i < CW; i += 2) y[i / 2] = pk(a[i], a[i + 1]);
      if (NA == 2) {
        float b[CW];
        tmem_ld_async(s_addr(it, 1), b);
        tmem_ld_wait(b);
        const u64 ps = pk(1.f / kPartScale, 1.f / kPartScale);
#pragma unroll
        for (int i = 0; i < CW; i += 2) y[i / 2] = fma2(pk(b[i], b[i + 1]), ps, y[i / 2]);
      }
#pragma unroll
      for (int i = 0; i < CW; i += 4) {
        const ulonglong2 r = *reinterpret_cast<const ulonglong2*>(rf + c0 + i);
        const u64 f0 = mul2(r.x, kf2), f1 = mul2(r.y, kf2);
        if (ref) {
          y[i / 2] = mul2(y[i / 2], f0);
          y[i / 2 + 1] = mul2(y[i / 2 + 1], f1);
        } else {
          const ulonglong2 m = *reinterpret_cast<const ulonglong2*>(nm + c0 + i);
          y[i / 2] = fma2(y[i / 2], f0, m.x);
          y[i / 2 + 1] = fma2(y[i / 2 + 1], f1, m.y);
        }
      }
    };
#pragma unroll 1
    for (int it = 0; it < n; ++it) {
      if (fresh) {
        // ---- a KV head begins: its queries, in parts (the S MMAs that read
        // the previous head's are done: this thread has waited for them)
        pend1 = pend2 = false;
        E = 1024;  // (none yet: the first tile's takes its place)
#pragma unroll
        for (int i = 0; i < CW / 2; ++i) l[i] = o[i] = 0ull;
        const size_t q0 = ((static_cast<size_t>(pos.s) * d.Hq + pos.g * d.G) * d.B + r0) * kD;
        // (all of the warp's rows in flight at once)
        float4 xr[NR / W0];
#pragma unroll
        for (int i = 0; i < NR / W0; ++i) {
          const int r = warp + i * W0;
          xr[i] = r < nrows ? ld4(Q, q0 + static_cast<size_t>(r) * kD + 4 * lane,
                                  NQ == 2 ? LOSA_BF16 : LOSA_F32)
                            : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        bar_sync(5, NS);
#pragma unroll
        for (int i = 0; i < NR / W0; ++i) {
          const int r = warp + i * W0;
          float4 x = xr[i];
          const float amax = warp_max(fmaxf(fmaxf(fabsf(x.x), fabsf(x.y)), fmaxf(fabsf(x.z), fabsf(x.w))));
          const int c = 7 - max(static_cast<int>(__float_as_uint(amax) >> 23) - 127, -119);
          const float sc = exp2_int(c);
          x = make_float4(x.x * sc, x.y * sc, x.z * sc, x.w * sc);
          char* dst = qs + r * 128 + (((lane >> 2) ^ (r & 7)) << 4) + (lane & 3) * 4;
#pragma unroll
          for (int p = 0; p < NQ; ++p) {
            // (an infinite row maximum leaves no number: NaN, as its softmax)
            const uint32_t w = amax == INFINITY          ? 0x7f7f7f7fu
                               : NQ == 2 && p == 1 ? e5m2x4(x.x, x.y, x.z, x.w)
                                                   : e4m3x4(x.x, x.y, x.z, x.w);
            *reinterpret_cast<uint32_t*>(dst + p * NR * kD) = w;
            if (p == NQ - 1) break;
            const float4 y = e4m3x4_to_f32(w);
            const float f = NA == 2 && p == NQ / 2 - 1 ? kPartScale : 1.f;
            x = make_float4((x.x - y.x) * f, (x.y - y.y) * f, (x.z - y.z) * f, (x.w - y.w) * f);
          }
          if (lane == 0) {
            rf[r] = amax < INFINITY ? exp2_int(-c) : 1.f;
            nm[r] = INFINITY;
          }
        }
        fence_async_smem();
        bar_sync(5, NS);
        if (lane == 0) mbar_arrive(bQ);
      }
      // S^T of this tile and all MMAs issued before it are done: O = V W of two
      // tiles back too, so that may be read and W's buffer of this parity is free
      mbar_wait_or(&bS[it & 1], (it >> 1) & 1, s_fail);
      __syncwarp();
      tc_fence_after();
      float sc[CW];
      tmem_ld_async(s_addr(it, 0), sc);
      const float4 pg = info[it & 1].page[key >> 4];
      const int nv = __float_as_int(pg.w) & 255;
      const bool last = __float_as_int(pg.w) >= 256;
      const bool valid = key < nv;
      const int new_e = __float_as_int(pg.z);
      const u64 kf2 = pk(pg.x, pg.x), vs2 = pk(pg.y, pg.y);
      if (pend2) take_o(it & 1);
      tmem_ld_wait(sc);
      u64 y[CW / 2];
      to_x(it, kf2, false, sc, y);
      float top = -INFINITY;
#pragma unroll
      for (int i = 0; i < CW; i += 4) {
        const float2 a = up(y[i / 2]), b = up(y[i / 2 + 1]);
        top = max3(max3(top, a.x, a.y), b.x, b.y);
      }
      pend2 = pend1;
      if (bar_or(1 + wg, 128, (valid && top > kRefMove) || new_e != E)) {
        // ---- some row's reference or E moves (the first tile; then seldom): the
        // columns' maxima over the tile's keys, references, and what has been
        // accumulated against the old ones
        tmem_ld_async(s_addr(it, 0), sc);
        tmem_ld_wait(sc);
        to_x(it, kf2, true, sc, y);
        float mine = -INFINITY;
#pragma unroll
        for (int i = 0; i < CW; i += 2) {
          const float2 a = up(y[i / 2]);
          const float m0 = redux_max(valid ? a.x : -INFINITY);
          const float m1 = redux_max(valid ? a.y : -INFINITY);
          if (lane == i) mine = m0;
          if (lane == i + 1) mine = m1;
        }
        if (lane < CW) xg[w4 * CW + lane] = mine;
        bar_sync(1 + wg, 128);
        if (w4 == 0 && lane < CW) {
          float m = mine;
#pragma unroll
          for (int w = 1; w < 4; ++w) m = fmaxf(m, xg[w * CW + lane]);
          const float old = -nm[c0 + lane];
          const bool move = m > old + kRefMove || (old == -INFINITY && m > old);
          const float ref = move ? m : old;
          ag[lane] = move ? exp2f(old - ref) : 1.f;
          nm[c0 + lane] = -ref;
        }
        bar_sync(1 + wg, 128);
        if (pend2) {  // the tile before's product, against the old references too
          mbar_wait_or(&bO[(it - 1) & 1], ((it - 1) >> 1) & 1, s_fail);
          __syncwarp();
          tc_fence_after();
          take_o((it - 1) & 1);
          pend2 = false;
        }
        const float f = exp2_int(max(min(E - new_e, 0), -126));
        const u64 f2 = pk(f, f);
        E = new_e;
#pragma unroll
        for (int i = 0; i < CW; i += 2) {
          const u64 a = *reinterpret_cast<const u64*>(ag + i);
          o[i / 2] = mul2(mul2(o[i / 2], a), f2);
          l[i / 2] = mul2(l[i / 2], a);
          y[i / 2] = add2(y[i / 2], *reinterpret_cast<const u64*>(nm + c0 + i));
        }
        // (the next vote's slow path writes xch, nm and alpha only after a
        // barrier of this warp group)
      }
      pend1 = true;
      if (nv < kLineKeys) {
        const u64 none = pk(-INFINITY, -INFINITY);
#pragma unroll
        for (int i = 0; i < CW / 2; ++i) y[i] = valid ? y[i] : none;
      }
      char* wrow = wbuf + (it & 1) * C::wbytes + key * 128;
#pragma unroll
      for (int i = 0; i < CW; i += 8) {
        uint32_t hi[4], mid[4], lo[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const float2 a = up(y[i / 2 + u]);
          const u64 p = pk(ex2_approx(a.x), ex2_approx(a.y));
          l[i / 2 + u] = add2(l[i / 2 + u], p);
          const float2 w = up(mul2(p, vs2));
          // cut off, not rounded: what a part leaves is exact; mid is stored negated
          hi[u] = bf16x2_top(w);
          const float2 r = bf16x2_sub(hi[u], w);
          mid[u] = bf16x2_top(r);
          lo[u] = bf16x2_top(bf16x2_sub(mid[u], r));
        }
        // the 16-byte chunk of these columns in the key's row
        char* dst = wrow + ((((c0 + i) >> 3) ^ (key & 7)) << 4);
        *reinterpret_cast<uint4*>(dst) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<uint4*>(dst + C::atom) = make_uint4(mid[0], mid[1], mid[2], mid[3]);
        *reinterpret_cast<uint4*>(dst + 2 * C::atom) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
      }
      fence_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bP[it & 1]);
      fresh = last;

      if (last) {
        // ---- the KV head ends here: the partial of its rows
        mbar_wait_or(&bO[it & 1], (it >> 1) & 1, s_fail);  // (in order: the tile before's too)
        __syncwarp();
        tc_fence_after();
        const int sg = pos.s * d.Hkv + pos.g;
        float* dst0 = part + ((static_cast<size_t>(blockIdx.x) + sg) * rows + r0) * kPartStride;
        if (pend2) take_o((it - 1) & 1);
        take_o(it & 1);
        // sums over the lanes: after the exchange of halves, lane i / (32 / CW)
        // holds column i's
        float v[CW];
#pragma unroll
        for (int i = 0; i < CW; i += 2) {
          const float2 a = up(l[i / 2]);
          v[i] = a.x;
          v[i + 1] = a.y;
        }
        int w = CW;
#pragma unroll
        for (int sh = 16; sh > 0; sh >>= 1) {
          if (w > 1) {
            w >>= 1;
            const bool hi = lane & sh;
#pragma unroll
            for (int i = 0; i < CW / 2; ++i) {
              if (i < w) {
                const float send = hi ? v[i] : v[i + w], keep = hi ? v[i + w] : v[i];
                v[i] = keep + __shfl_xor_sync(0xffffffffu, send, sh);
              }
            }
          } else {
            v[0] += __shfl_xor_sync(0xffffffffu, v[0], sh);
          }
        }
        bar_sync(1 + wg, 128);  // (xch: the maxima have been read)
        if (lane % (32 / CW) == 0) xg[w4 * CW + lane / (32 / CW)] = v[0];
        bar_sync(1 + wg, 128);
        const bool good = *s_fail == 0;
#pragma unroll
        for (int i = 0; i < CW; i += 2) {
          const float2 a = up(o[i / 2]);
          if (good && c0 + i < nrows) dst0[(c0 + i) * kPartStride + 4 + key] = a.x;
          if (good && c0 + i + 1 < nrows) dst0[(c0 + i + 1) * kPartStride + 4 + key] = a.y;
        }
        if (good && w4 == 0 && lane < CW && c0 + lane < nrows) {
          float sum = 0.f;
#pragma unroll
          for (int q = 0; q < 4; ++q) sum += xg[q * CW + lane];
          float* dst = dst0 + (c0 + lane) * kPartStride;
          dst[0] = -nm[c0 + lane];
          dst[1] = sum;
          dst[2] = __int_as_float(E);
        }
        pos.next_head(d);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (tid == 0 && *s_fail) atomicCAS(status, 0, LOSA_ERR_DEVICE_TIMEOUT);
  if (warp == 1) tmem_dealloc(tb, C::cols);
}

template <int NR, int NQ>
int launch_partials(const Dims& d, const void* q, const void* k8, const void* v8,
                    const float* k_scale, const float* v_scale, float* part, int* status,
                    cudaStream_t st) {
  using C = QPlan<NR, NQ>;
  auto* fn = dense_quant_kernel<NR, NQ>;
  static DeviceOnce<kMaxDevices> attrs;
  int dev = 0;
  cudaGetDevice(&dev);
  const cudaError_t e = attrs.run(dev, [&] {
    return cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, C::smem);
  });
  if (e != cudaSuccess) return record_cuda_error(e);
  CUtensorMap kmap, vmap;
  const unsigned long long nrows = static_cast<unsigned long long>(d.S) * d.Hkv * d.Lc;
  if (make_byte_tmap(&kmap, k8, nrows, kLineKeys) != LOSA_OK ||
      make_byte_tmap(&vmap, v8, nrows, kLineKeys) != LOSA_OK)
    return record_cuda_error(cudaErrorInvalidValue);
  return launch_behind(fn, dim3(d.line_ctas, (d.G * d.B + NR - 1) / NR), C::threads, C::smem, st, q,
                       kmap, vmap, k_scale, v_scale, part, status, d);
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
  // (the tensor maps' row coordinate is an int)
  if (SG > 65535 || SG * d.Lc > 0x7fffffffu) return LOSA_ERR_UNSUPPORTED;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  float* part = reinterpret_cast<float*>(static_cast<char*>(workspace) + d.off_part);
  int* status = reinterpret_cast<int*>(static_cast<char*>(workspace) + d.off_status);
  // the fewest columns that hold the rows: what a tile costs beyond its loads
  // grows with them (8 KV heads, 64K prefix, 16 rows: 31.2 us with 16 columns,
  // 35.1 with 32, 45.4 with 64; fp32 38.4, 40.7, 52.1)
  const int r = d.G * d.B;
  auto* launch = d.dtype == LOSA_BF16 ? (r <= 16   ? launch_partials<16, 2>
                                         : r <= 32 ? launch_partials<32, 2>
                                                   : launch_partials<64, 2>)
                                      : (r <= 16   ? launch_partials<16, 6>
                                         : r <= 32 ? launch_partials<32, 6>
                                                   : launch_partials<64, 6>);
  rc = launch(d, q, k8, v8, k_scale, v_scale, part, status, st);
  if (rc != LOSA_OK) return rc;
  return launch_dense_finish(d, q, k_blk, v_blk, part, o_p, l_p, out, out_lse, st);
}
