// The 4-bit cache: entries written, read back and evicted. The page format is in int4.cuh, the
// attention over it in int4_attend.cu.
//
//   qe_int4_append  quantises new tokens' keys and values into their units' next entries
//   qe_int4_read    the values that entries stand for
//   qe_int4_evict   keeps the newest entries and those of highest accumulated attention weight
//                   ("Resumo Técnico: QEvict", Pontuação Cumulativa, entry by entry)
#include "int4.cuh"
#include "warp_mma.cuh"

namespace {

constexpr int kRowThreads = 256;

struct RowArgs {
  const void* k;
  const void* v;
  void* k_out;
  void* v_out;
  long long ks, vs;       // elements between tokens
  const int32_t* cu;      // [B + 1]
  const int32_t* first;   // read: [U] first entry, or null
  const float* mass;      // append: [T][Hkv], or null
  int T;
};

// Whether every bound is in order (0 <= cu[b] <= cu[b + 1] <= T); the first bad b is recorded.
// Called by a whole warp.
__device__ bool bounds_ok(const int32_t* cu, int B, int T, int32_t* status) {
  const int lane = threadIdx.x & 31;
  int bad = 0x7fffffff;
  for (int b = lane; b < B; b += 32)
    if (cu[b] < 0 || cu[b + 1] < cu[b] || cu[b + 1] > T) bad = min(bad, b);
  bad = __reduce_min_sync(0xffffffffu, bad);
  if (bad != 0x7fffffff && lane == 0) qe_record_error(status, QE_ERR_INVALID_ARG, bad);
  return bad == 0x7fffffff;
}

// the sequence b with cu[b] <= t < cu[b + 1], or -1 (bounds in order)
__device__ __forceinline__ int sequence_of(const int32_t* cu, int B, int t) {
  int lo = 0, hi = B;                     // cu[lo] <= t, cu[hi] > t
  if (t < cu[0] || t >= cu[B]) return -1;
  while (hi - lo > 1) {
    const int m = (lo + hi) >> 1;
    if (cu[m] <= t) lo = m; else hi = m;
  }
  return lo;
}

// An item is one token of one kv head, a key row and a value row of D elements: D / 4 lanes take
// four consecutive elements of each, so a group of 32 is eight lanes.
template <typename T, int D>
__global__ void __launch_bounds__(kRowThreads) int4_append_kernel(Int4View c, RowArgs a) {
  constexpr int LPI = D / 4, NG = D / 32, IPB = kRowThreads / LPI;
  __shared__ int s_ok;
  if (threadIdx.x < 32) {
    const bool ok = bounds_ok(a.cu, c.B, a.T, c.status);
    if (threadIdx.x == 0) s_ok = ok;
  }
  __syncthreads();
  if (!s_ok) return;
  const int sub = threadIdx.x / LPI, l = threadIdx.x % LPI, g = l / 8, e8 = l % 8;
  const long long items = (long long)a.T * c.Hkv;
  for (long long it0 = (long long)blockIdx.x * IPB; it0 < items; it0 += (long long)gridDim.x * IPB) {
    const long long it = it0 + sub;
    const bool live = it < items;
    const int t = live ? (int)(it / c.Hkv) : 0, h = live ? (int)(it % c.Hkv) : 0;
    float k[4] = {}, v[4] = {};
    if (live) {
      const uint2 kw = *reinterpret_cast<const uint2*>(static_cast<const T*>(a.k) + t * a.ks + h * D + 4 * l);
      const uint2 vw = *reinterpret_cast<const uint2*>(static_cast<const T*>(a.v) + t * a.vs + h * D + 4 * l);
      k[0] = Elem<T>::lo(kw.x), k[1] = Elem<T>::hi(kw.x), k[2] = Elem<T>::lo(kw.y), k[3] = Elem<T>::hi(kw.y);
      v[0] = Elem<T>::lo(vw.x), v[1] = Elem<T>::hi(vw.x), v[2] = Elem<T>::lo(vw.y), v[3] = Elem<T>::hi(vw.y);
    }
    float kmn = fminf(fminf(k[0], k[1]), fminf(k[2], k[3])), kmx = fmaxf(fmaxf(k[0], k[1]), fmaxf(k[2], k[3]));
    float vmn = fminf(fminf(v[0], v[1]), fminf(v[2], v[3])), vmx = fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3]));
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) {
      kmn = fminf(kmn, __shfl_xor_sync(0xffffffffu, kmn, o));
      kmx = fmaxf(kmx, __shfl_xor_sync(0xffffffffu, kmx, o));
      vmn = fminf(vmn, __shfl_xor_sync(0xffffffffu, vmn, o));
      vmx = fmaxf(vmx, __shfl_xor_sync(0xffffffffu, vmx, o));
    }
    if (!live) continue;
    const int b = sequence_of(a.cu, c.B, t);
    if (b < 0) continue;                                  // rows outside every sequence
    const int u = b * c.Hkv + h, n = a.cu[b + 1] - a.cu[b], j = t - a.cu[b];
    const int len = c.lengths[u];
    if (len < 0 || (long long)len + n > (long long)c.max_pages * kInt4Page) {
      if (l == 0) qe_record_error(c.status, len < 0 ? QE_ERR_INVALID_ARG : QE_ERR_POOL_EXHAUSTED, u);
      continue;
    }
    const int e = len + j, i = e % kInt4Page;
    const int page = c.table[(size_t)u * c.max_pages + e / kInt4Page];
    if (page < 0 || page >= c.n_pages) {
      if (l == 0) qe_record_error(c.status, QE_ERR_DEVICE_FAULT, u);
      continue;
    }
    const Int4Group kg(kmn, kmx), vg(vmn, vmx);
    uint32_t kc = 0, vc = 0;
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      kc |= kg.code(k[x]) << (4 * x);
      vc |= vg.code(v[x]) << (4 * x);
    }
    uint8_t* pg = c.pages + (size_t)page * (20 * D);
    *reinterpret_cast<uint16_t*>(pg + i * (D / 2) + ((e8 >> 1) * NG + g) * 4 + (e8 & 1) * 2) = (uint16_t)kc;
    *reinterpret_cast<uint16_t*>(pg + 8 * D + i * (D / 2) + (e8 * NG + g) * 2) = (uint16_t)vc;
    if (e8 == 0) {
      __half* m = reinterpret_cast<__half*>(pg + 16 * D);
      const int km = i * NG + g, vm = ((((i & 7) >> 1) * NG + g) * 2 + (i >> 3)) * 2 + (i & 1);
      m[km] = kg.sh;
      m[D / 2 + km] = kg.zh;
      m[D + vm] = vg.sh;
      m[3 * D / 2 + vm] = vg.zh;
    }
    if (l == 0) {
      const size_t at = (size_t)page * kInt4Page + i;
      c.mass[at] = a.mass ? a.mass[(size_t)t * c.Hkv + h] : 0.f;
      c.pos[at] = c.seen[b] + j;
    }
  }
  // the last CTA to finish moves the lengths on: every other one has read them
  __shared__ int s_last;
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    s_last = atomicAdd(&c.status[2], 1) == (int)gridDim.x - 1;
  }
  __syncthreads();
  if (!s_last) return;
  for (int u = threadIdx.x; u < c.B * c.Hkv; u += blockDim.x) {
    const int b = u / c.Hkv, n = a.cu[b + 1] - a.cu[b], len = c.lengths[u];
    if (len >= 0 && (long long)len + n <= (long long)c.max_pages * kInt4Page) c.lengths[u] = len + n;
    if (u % c.Hkv == 0) c.seen[b] += n;
  }
  if (threadIdx.x == 0) c.status[2] = 0;
}

template <typename T, int D>
__global__ void __launch_bounds__(kRowThreads) int4_read_kernel(Int4View c, RowArgs a) {
  constexpr int LPI = D / 4, NG = D / 32, IPB = kRowThreads / LPI;
  __shared__ int s_ok;
  if (threadIdx.x < 32) {
    const bool ok = bounds_ok(a.cu, c.B, a.T, c.status);
    if (threadIdx.x == 0) s_ok = ok;
  }
  __syncthreads();
  if (!s_ok) return;
  const int sub = threadIdx.x / LPI, l = threadIdx.x % LPI, g = l / 8, e8 = l % 8;
  const long long items = (long long)a.T * c.Hkv;
  for (long long it = (long long)blockIdx.x * IPB + sub; it < items; it += (long long)gridDim.x * IPB) {
    const int t = (int)(it / c.Hkv), h = (int)(it % c.Hkv);
    const int b = sequence_of(a.cu, c.B, t);
    if (b < 0) continue;
    const int u = b * c.Hkv + h;
    const long long e = (long long)(a.first ? a.first[u] : 0) + t - a.cu[b];
    if (e < 0 || e >= c.lengths[u] || e >= (long long)c.max_pages * kInt4Page) continue;   // no such entry
    const int i = (int)(e % kInt4Page), page = c.table[(size_t)u * c.max_pages + e / kInt4Page];
    if (page < 0 || page >= c.n_pages) {
      if (l == 0) qe_record_error(c.status, QE_ERR_DEVICE_FAULT, u);
      continue;
    }
    const uint8_t* pg = c.pages + (size_t)page * (20 * D);
    const uint32_t kc = *reinterpret_cast<const uint16_t*>(pg + i * (D / 2) + ((e8 >> 1) * NG + g) * 4 + (e8 & 1) * 2);
    const uint32_t vc = *reinterpret_cast<const uint16_t*>(pg + 8 * D + i * (D / 2) + (e8 * NG + g) * 2);
    const __half* m = reinterpret_cast<const __half*>(pg + 16 * D);
    const int km = i * NG + g, vm = ((((i & 7) >> 1) * NG + g) * 2 + (i >> 3)) * 2 + (i & 1);
    const float ksc = __half2float(m[km]), kz = __half2float(m[D / 2 + km]);
    const float vsc = __half2float(m[D + vm]), vz = __half2float(m[3 * D / 2 + vm]);
    // c s is exact in float32; the sum is rounded to float32, then to the output type
    T ko[4], vo[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      ko[x] = Elem<T>::from_f(fmaf((float)(kc >> (4 * x) & 15u), ksc, kz));
      vo[x] = Elem<T>::from_f(fmaf((float)(vc >> (4 * x) & 15u), vsc, vz));
    }
    const size_t o = ((size_t)t * c.Hkv + h) * D + 4 * l;
    *reinterpret_cast<uint2*>(static_cast<T*>(a.k_out) + o) = *reinterpret_cast<uint2*>(ko);
    *reinterpret_cast<uint2*>(static_cast<T*>(a.v_out) + o) = *reinterpret_cast<uint2*>(vo);
  }
}

// ---------------------------------------------------------------------------------------
// eviction
// ---------------------------------------------------------------------------------------

constexpr int kSelThreads = 1024;

// Order of the entries: the newest ones above all, then by weight. A NaN weight is below every
// other; -0 equals +0.
__device__ __forceinline__ uint32_t evict_key(float w, bool newest) {
  if (newest) return 0xffffffffu;
  const uint32_t b = __float_as_uint(w);
  if (w != w) return 0u;
  if ((b << 1) == 0u) return 0x80000000u;
  return (b >> 31) ? ~b : (b | 0x80000000u);
}

// The survivors of one unit, a CTA each: the budget-th highest key T by a radix select, the entries
// above it, and of those equal to it the first ones. Their indices go, in order, to the pos slots
// of their new places (the move kernel puts the positions there).
__global__ void __launch_bounds__(kSelThreads) int4_select_kernel(Int4View s, Int4View d, int budget, int recent) {
  __shared__ uint32_t hist[256];
  __shared__ uint32_t ctl[2];
  __shared__ int wsum[2][32];
  __shared__ int base[2];
  const int u = blockIdx.x, b = u / s.Hkv, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int32_t* table = s.table + (size_t)u * s.max_pages;
  const int32_t* dtable = d.table + (size_t)u * d.max_pages;
  int len = s.lengths[u];
  if (tid == 0 && u % s.Hkv == 0) d.seen[b] = s.seen[b];
  if (len < 0 || (long long)len > (long long)s.max_pages * kInt4Page) {
    if (tid == 0) {
      qe_record_error(s.status, QE_ERR_INVALID_ARG, u);
      d.lengths[u] = 0;
    }
    return;
  }
  const long long cut = (long long)s.seen[b] - recent;
  auto key_of = [&](int e) -> uint32_t {
    const int page = table[e / kInt4Page];
    if (page < 0 || page >= s.n_pages) return 0u;
    const size_t at = (size_t)page * kInt4Page + e % kInt4Page;
    return evict_key(s.mass[at], s.pos[at] >= cut);
  };
  const int keep = min(len, budget);
  uint32_t T = 0;         // keys above T are kept,
  int ties = len;         // and the first `ties` equal to it
  if (len > budget) {
    uint32_t prefix = 0, mask = 0;
    int k = budget;
    for (int sh = 24; sh >= 0; sh -= 8) {
      for (int x = tid; x < 256; x += kSelThreads) hist[x] = 0;
      __syncthreads();
      for (int e = tid; e < len; e += kSelThreads) {
        const uint32_t key = key_of(e);
        if ((key & mask) == prefix) atomicAdd(&hist[key >> sh & 255u], 1u);
      }
      __syncthreads();
      if (tid == 0) {
        int above = 0, x = 255;
        while (above + (int)hist[x] < k) above += hist[x--];
        ctl[0] = x;
        ctl[1] = above;
      }
      __syncthreads();
      prefix |= ctl[0] << sh;
      mask |= 255u << sh;
      k -= ctl[1];
      __syncthreads();
    }
    T = prefix;
    ties = k;
  }
  if (tid < 2) base[tid] = 0;
  __syncthreads();
  for (int e0 = 0; e0 < len; e0 += kSelThreads) {
    const int e = e0 + tid;
    const uint32_t key = e < len ? key_of(e) : 0u;
    const bool eq = e < len && (len <= budget || key == T), gt = e < len && len > budget && key > T;
    const uint32_t beq = __ballot_sync(0xffffffffu, eq), bgt = __ballot_sync(0xffffffffu, gt);
    if (lane == 0) wsum[0][warp] = __popc(beq), wsum[1][warp] = __popc(bgt);
    __syncthreads();
    if (warp == 0) {
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        const int own = wsum[w][lane];
        int inc = own;
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, inc, o);
          if (lane >= o) inc += y;
        }
        wsum[w][lane] = base[w] + inc - own;
        __syncwarp();
        if (lane == 31) base[w] += inc;
      }
    }
    __syncthreads();
    const uint32_t below = (1u << lane) - 1u;
    const int neq = wsum[0][warp] + __popc(beq & below), ngt = wsum[1][warp] + __popc(bgt & below);
    if (gt || (eq && neq < ties)) {
      const int to = ngt + min(neq, ties);
      const int page = dtable[to / kInt4Page];
      if (page < 0 || page >= d.n_pages)
        qe_record_error(d.status, QE_ERR_DEVICE_FAULT, u);
      else
        d.pos[(size_t)page * kInt4Page + to % kInt4Page] = e;
    }
    __syncthreads();
  }
  if (tid == 0) d.lengths[u] = keep;
}

// One warp assembles one destination page: the records of its entries, their weights and positions.
// Slots behind the unit's last entry are left as they were.
template <int D>
__global__ void __launch_bounds__(128) int4_move_kernel(Int4View s, Int4View d, int pages_per_unit) {
  constexpr int NG = D / 32, RV = D / 32;   // 16-byte pieces of a row of codes
  const int wid = blockIdx.x * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int u = wid / pages_per_unit, p = wid % pages_per_unit;
  if (u >= d.B * d.Hkv) return;
  const int live = min(kInt4Page, d.lengths[u] - p * kInt4Page);
  if (live <= 0) return;
  const int dp = d.table[(size_t)u * d.max_pages + p];
  if (dp < 0 || dp >= d.n_pages) return;    // recorded by the selection
  // lane i < 16 holds where entry i comes from: its page and slot
  int sp = -1, ss = 0;
  const size_t at = (size_t)dp * kInt4Page + lane;
  if (lane < live) {
    const int e = d.pos[at];
    const bool in = e >= 0 && e < s.max_pages * kInt4Page;   // holds unless tables share a page
    sp = !in ? -1 : s.table[(size_t)u * s.max_pages + e / kInt4Page];
    ss = e % kInt4Page;
    if (sp < 0 || sp >= s.n_pages) {
      qe_record_error(s.status, QE_ERR_DEVICE_FAULT, u);
      sp = -1;
    }
    if (sp >= 0) {
      const size_t from = (size_t)sp * kInt4Page + ss;
      d.mass[at] = s.mass[from];
      d.pos[at] = s.pos[from];
    }
  }
  uint8_t* dst = d.pages + (size_t)dp * (20 * D);
#pragma unroll
  for (int part = 0; part < 2; ++part)      // K and V codes
#pragma unroll
    for (int x = 0; x < 16 * RV; x += 32) {
      const int i = (x + lane) / RV, o = ((x + lane) % RV) * 16;
      const int fp = __shfl_sync(0xffffffffu, sp, i), fs = __shfl_sync(0xffffffffu, ss, i);
      if (fp >= 0)
        *reinterpret_cast<uint4*>(dst + part * 8 * D + i * (D / 2) + o) = *reinterpret_cast<const uint4*>(
            s.pages + (size_t)fp * (20 * D) + part * 8 * D + fs * (D / 2) + o);
    }
#pragma unroll
  for (int x = 0; x < 16 * NG; x += 32) {   // metadata: a half of each of the four kinds
    const int i = (x + lane) / NG, g = (x + lane) % NG;
    const int fp = __shfl_sync(0xffffffffu, sp, i), fs = __shfl_sync(0xffffffffu, ss, i);
    if (fp >= 0) {
      const uint16_t* from = reinterpret_cast<const uint16_t*>(s.pages + (size_t)fp * (20 * D) + 16 * D);
      uint16_t* to = reinterpret_cast<uint16_t*>(dst + 16 * D);
      const int fk = fs * NG + g, tk = i * NG + g;
      const int fv = ((((fs & 7) >> 1) * NG + g) * 2 + (fs >> 3)) * 2 + (fs & 1);
      const int tv = ((((i & 7) >> 1) * NG + g) * 2 + (i >> 3)) * 2 + (i & 1);
      to[tk] = from[fk];
      to[D / 2 + tk] = from[D / 2 + fk];
      to[D + tv] = from[D + fv];
      to[3 * D / 2 + tv] = from[3 * D / 2 + fv];
    }
  }
}

int sm_count(int* sms) {
  static QeOnce once;
  static int of[QE_MAX_DEVICES];
  int dev = 0;
  const int e = qe_once_per_device(once, &dev, [&](int d) {
    QE_CUDA_TRY(cudaDeviceGetAttribute(&of[d], cudaDevAttrMultiProcessorCount, d));
    return QE_OK;
  });
  if (e == QE_OK) *sms = of[dev];
  return e;
}

}  // namespace

int int4_view(const qe_int4_cache* c, Int4View* v) {
  if (!c || !c->pages || !c->page_table || !c->lengths || !c->seen || !c->mass || !c->pos || !c->status)
    return QE_ERR_INVALID_ARG;
  if (c->B < 1 || c->Hkv < 1 || c->max_pages < 1 || c->n_pages < 1 || !qe_aligned(c->pages, 16))
    return QE_ERR_INVALID_ARG;
  if (c->D != 64 && c->D != 128) return QE_ERR_UNSUPPORTED_SHAPE;
  if ((long long)c->B * c->Hkv * c->max_pages * kInt4Page >= (1ll << 31)) return QE_ERR_UNSUPPORTED_SHAPE;
  *v = Int4View{static_cast<uint8_t*>(c->pages), c->page_table, c->lengths, c->seen, c->mass,
                c->pos, c->status, c->B, c->Hkv, c->max_pages, c->n_pages};
  return QE_OK;
}

QE_API int qe_int4_append(const qe_int4_cache* cache, const void* k, const void* v, long long k_stride,
                          long long v_stride, const int32_t* cu_seqlens, int T, int dtype, const float* mass,
                          qe_stream_t stream) {
  Int4View c;
  int e = int4_view(cache, &c);
  if (e) return e;
  if (T < 0 || !cu_seqlens || (dtype != QE_FP16 && dtype != QE_BF16)) return QE_ERR_INVALID_ARG;
  if (T == 0) return QE_OK;
  const int D = cache->D;
  if (!k || !v || !qe_aligned(k, 8) || !qe_aligned(v, 8) || k_stride < (long long)c.Hkv * D ||
      v_stride < (long long)c.Hkv * D || k_stride % 4 || v_stride % 4)
    return QE_ERR_INVALID_ARG;
  int sms = 0;
  if ((e = sm_count(&sms))) return e;
  RowArgs a{};
  a.k = k, a.v = v, a.ks = k_stride, a.vs = v_stride, a.cu = cu_seqlens, a.mass = mass, a.T = T;
  const long long per = kRowThreads / (D / 4), want = ((long long)T * c.Hkv + per - 1) / per;
  const int grid = (int)(want < 8ll * sms ? want : 8ll * sms);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const bool bf = dtype == QE_BF16;
  if (D == 128) {
    if (bf) int4_append_kernel<__nv_bfloat16, 128><<<grid, kRowThreads, 0, st>>>(c, a);
    else int4_append_kernel<__half, 128><<<grid, kRowThreads, 0, st>>>(c, a);
  } else {
    if (bf) int4_append_kernel<__nv_bfloat16, 64><<<grid, kRowThreads, 0, st>>>(c, a);
    else int4_append_kernel<__half, 64><<<grid, kRowThreads, 0, st>>>(c, a);
  }
  return cudaGetLastError() == cudaSuccess ? QE_OK : QE_ERR_CUDA;
}

QE_API int qe_int4_read(const qe_int4_cache* cache, const int32_t* cu_seqlens, int T, const int32_t* first, int dtype,
                        void* k_out, void* v_out, qe_stream_t stream) {
  Int4View c;
  int e = int4_view(cache, &c);
  if (e) return e;
  if (T < 0 || !cu_seqlens || (dtype != QE_FP16 && dtype != QE_BF16)) return QE_ERR_INVALID_ARG;
  if (T == 0) return QE_OK;
  if (!k_out || !v_out || !qe_aligned(k_out, 8) || !qe_aligned(v_out, 8)) return QE_ERR_INVALID_ARG;
  int sms = 0;
  if ((e = sm_count(&sms))) return e;
  const int D = cache->D;
  RowArgs a{};
  a.k_out = k_out, a.v_out = v_out, a.cu = cu_seqlens, a.first = first, a.T = T;
  const long long per = kRowThreads / (D / 4), want = ((long long)T * c.Hkv + per - 1) / per;
  const int grid = (int)(want < 8ll * sms ? want : 8ll * sms);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const bool bf = dtype == QE_BF16;
  if (D == 128) {
    if (bf) int4_read_kernel<__nv_bfloat16, 128><<<grid, kRowThreads, 0, st>>>(c, a);
    else int4_read_kernel<__half, 128><<<grid, kRowThreads, 0, st>>>(c, a);
  } else {
    if (bf) int4_read_kernel<__nv_bfloat16, 64><<<grid, kRowThreads, 0, st>>>(c, a);
    else int4_read_kernel<__half, 64><<<grid, kRowThreads, 0, st>>>(c, a);
  }
  return cudaGetLastError() == cudaSuccess ? QE_OK : QE_ERR_CUDA;
}

QE_API int qe_int4_evict(const qe_int4_cache* src, const qe_int4_cache* dst, int budget, int recent,
                         qe_stream_t stream) {
  Int4View s, d;
  int e = int4_view(src, &s);
  if (e || (e = int4_view(dst, &d))) return e;
  if (src->B != dst->B || src->Hkv != dst->Hkv || src->D != dst->D) return QE_ERR_INVALID_ARG;
  if (budget < 1 || recent < 0 || budget > (long long)d.max_pages * kInt4Page) return QE_ERR_INVALID_ARG;
  if (s.pages == d.pages || s.lengths == d.lengths || s.seen == d.seen || s.mass == d.mass || s.pos == d.pos)
    return QE_ERR_INVALID_ARG;
  const int U = s.B * s.Hkv, ppu = (budget + kInt4Page - 1) / kInt4Page;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  int4_select_kernel<<<U, kSelThreads, 0, st>>>(s, d, budget, recent);
  const int grid = (int)(((long long)U * ppu + 3) / 4);
  if (src->D == 128) int4_move_kernel<128><<<grid, 128, 0, st>>>(s, d, ppu);
  else int4_move_kernel<64><<<grid, 128, 0, st>>>(s, d, ppu);
  return cudaGetLastError() == cudaSuccess ? QE_OK : QE_ERR_CUDA;
}
