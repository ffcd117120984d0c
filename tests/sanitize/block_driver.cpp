// Sanitizer driver for the host code of the block's operators: every entry
// point of include/gdn_block.h over a grid of problems that must pass (the
// launch stubs check every device pointer against the regions handed in).
// Device pointers are fake, well-separated addresses.  Exits non-zero on any
// failed expectation.
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include <initializer_list>

#include "gdn_block.h"
#include "sanitize_regions.h"

namespace {

int g_fail = 0;
long g_cases = 0;

void expect(bool ok, const char* what, int line, long code) {
  ++g_cases;
  if (!ok && ++g_fail < 30) fprintf(stderr, "FAIL line %d: %s (%ld)\n", line, what, code);
}
#define EXPECT(cond, code) expect(cond, #cond, __LINE__, (long)(code))

struct Fake {
  int slot = 0;
  template <typename T = void>
  T* take(int64_t bytes, int64_t off = 0) {
    if (bytes <= 0) return nullptr;
    const uintptr_t p = (uintptr_t(1) << 44) + (uintptr_t)(slot++) * (uintptr_t(1) << 40) + off;
    sanitize_region(reinterpret_cast<void*>(p), bytes);
    return reinterpret_cast<T*>(p);
  }
};

void done(int code, int calls) {
  EXPECT(code == GDN_OK, code);
  EXPECT(sanitize_calls() == calls, sanitize_calls());
  EXPECT(sanitize_violations() == 0, sanitize_violations());
}

void pack(int B, int L, int H, int D, int io, int gap, int off) {
  const int64_t es = io == GDN_BF16 ? 2 : 4, w = (int64_t)H * D + gap, n = (int64_t)B * L * H;
  gdn_pack8_problem p;
  memset(&p, 0, sizeof p);
  p.B = B; p.L = L; p.H = H; p.D = D; p.io_dtype = io;
  p.stride[0] = L * w; p.stride[1] = w;
  for (int un = 0; un < 2; ++un) {
    sanitize_reset();
    Fake f;
    void* x = f.take(((int64_t)B * L * w - gap) * es, off * es);
    gdn_checkpoint c = {f.take(n * D), f.take(n)};
    done(un ? gdn_unpack8(&p, &c, x, nullptr) : gdn_pack8(&p, x, &c, nullptr), 1);
  }
}

void qk(int B, int L, int Hq, int Hk, int D, int io, int norm, int axes, int gap, int off,
        bool weights, bool packed, bool shared) {
  const int64_t es = io == GDN_BF16 ? 2 : 4, tokens = (int64_t)B * L;
  const int64_t W = (int64_t)(Hq + 2 * Hk) * D + gap, nq = tokens * Hq * D, nk = tokens * Hk * D;
  gdn_qk_problem p;
  memset(&p, 0, sizeof p);
  p.B = B; p.L = L; p.Hq = Hq; p.Hk = Hk; p.D = D; p.io_dtype = io; p.norm = norm;
  p.pairing = D % 8 ? GDN_PAIR_ADJACENT : GDN_PAIR_HALVES;
  p.axes = axes; p.theta = 1e4; p.shared_positions = shared;
  for (int i = 0; i < axes; ++i) p.axis_pairs[i] = axes == 1 ? D / 4 * 2 / 2 * 1 : D / 16;
  int pairs = 0;
  for (int i = 0; i < axes; ++i) pairs += p.axis_pairs[i];
  if (pairs % 2) p.axis_pairs[0] += p.axis_pairs[0] > 1 ? -1 : 1;
  int64_t* strides[] = {p.q_stride, p.k_stride, p.dq_stride, p.dk_stride};
  for (int64_t* s : strides) s[0] = L * W, s[1] = W;
  pairs = p.axis_pairs[0] + p.axis_pairs[1] + p.axis_pairs[2];
  for (int back = 0; back < 2; ++back) {
    if (packed && norm == GDN_NORM_NONE && back) continue;
    // heads beyond 128 need four elements' alignment of what is used
    const bool strided = back || !packed;
    const bool refused = D > 128 && (pairs % 4 || (strided && (gap % 4 || off % 4)));
    sanitize_reset();
    Fake f;
    char* qkv = f.take<char>(((int64_t)B * L * W) * es + 64, off * es);
    const void* q = packed ? nullptr : qkv;
    const void* k = packed ? nullptr : qkv + (int64_t)Hq * D * es;
    gdn_checkpoint c[2] = {{f.take(nq), f.take(tokens * Hq)}, {f.take(nk), f.take(tokens * Hk)}};
    const bool w = weights && norm != GDN_NORM_NONE;
    const float* wq = w ? f.take<float>(D * 4) : nullptr;
    const float* wk = w ? f.take<float>(D * 4) : nullptr;
    const int32_t* pos =
        axes ? f.take<int32_t>((shared ? (int64_t)L : tokens) * axes * 4) : nullptr;
    const int32_t* len = f.take<int32_t>(B * 4);
    void* yq = f.take(nq * es);
    void* yk = f.take(nk * es);
    int code;
    if (!back) {
      code = gdn_qk_forward(&p, q, k, packed ? c : nullptr, wq, wk, pos, len, yq, yk,
                            packed ? nullptr : c, nullptr);
    } else {
      size_t ws = 0;
      EXPECT(gdn_qk_workspace_size(&p, w, &ws) == GDN_OK, ws);
      char* d = f.take<char>(((int64_t)B * L * W) * es + 64, off * es);
      float* dw = w ? f.take<float>(2 * D * 4) : nullptr;
      void* wsp = f.take((int64_t)ws);
      code = gdn_qk_backward(&p, q, k, packed ? c : nullptr, wq, wk, pos, len, yq, yk, d,
                             d + (int64_t)Hq * D * es, dw, w ? dw + D : nullptr, wsp, ws, nullptr);
    }
    if (refused) EXPECT(code == GDN_ERR_MISALIGNED, code);
    else done(code, 1);
  }
}

void lrec(int B, int L, int C, int io, int flags, int gap, int off, bool states, bool saved) {
  const int64_t es = io == GDN_BF16 ? 2 : 4, n = (int64_t)B * L * C, W = 2 * (int64_t)C + gap;
  gdn_lrec_problem p;
  memset(&p, 0, sizeof p);
  p.B = B; p.L = L; p.C = C; p.io_dtype = io; p.flags = flags;
  int64_t* strides[] = {p.x_stride, p.gate_stride, p.dx_stride, p.dgate_stride};
  for (int64_t* s : strides) s[0] = L * W, s[1] = W;
  size_t fw = 0, bw = 0, sv = 0;
  EXPECT(gdn_lrec_workspace_size(&p, GDN_OP_FORWARD, &fw) == GDN_OK, fw);
  EXPECT(gdn_lrec_workspace_size(&p, GDN_OP_BACKWARD, &bw) == GDN_OK, bw);
  EXPECT(gdn_lrec_saved_size(&p, &sv) == GDN_OK, sv);
  for (int back = 0; back < 2; ++back) {
    sanitize_reset();
    Fake f;
    char* xz = f.take<char>((int64_t)B * L * W * es, off * es);
    const int32_t* len = f.take<int32_t>(B * 4);
    float* h0 = states ? f.take<float>((int64_t)B * C * 4) : nullptr;
    float* h1 = states ? f.take<float>((int64_t)B * C * 4) : nullptr;
    void* s = saved ? f.take((int64_t)sv) : nullptr;
    void* o = f.take(n * es);
    if (!back) {
      void* ws = f.take((int64_t)fw);
      done(gdn_lrec_forward(&p, xz, xz + C * es, len, h0, o, h1, s, ws, fw, nullptr), 1);
      if (L == 1 && states)
        done(gdn_lrec_step(&p, xz, xz + C * es, h0, o, nullptr), 2);
    } else {
      char* d = f.take<char>((int64_t)B * L * W * es, off * es);
      float* dh = states ? f.take<float>((int64_t)B * C * 4) : nullptr;
      void* ws = f.take((int64_t)bw);
      done(gdn_lrec_backward(&p, xz, xz + C * es, len, h0, o, h1, s, d, d + C * es, dh, ws, bw,
                             nullptr),
           saved ? 1 : 2);
    }
  }
}

}  // namespace

int main() {
  for (int io : {GDN_BF16, GDN_FP32}) {
    for (int D : {4, 16, 20, 72, 112, 128, 256})
      for (int gap : {0, 4, 64})
        for (int B : {1, 3})
          for (int L : {1, 7}) {
            pack(B, L, 5, D, io, D > 128 ? gap / 4 * 4 : gap, gap ? 4 : 0);
            for (int norm : {0, 1, 2})
              for (int axes : {0, 1, 3}) {
                if (axes && D / 16 * 3 < 1 && axes == 3) continue;
                for (int bits = 0; bits < 8; ++bits)
                  qk(B, L, 6, 2, D, io, norm, D < 16 && axes == 3 ? 0 : axes, gap,
                     gap == 4 ? 2 : 0, bits & 1, bits & 2, bits & 4);
              }
          }
    for (int C : {1, 2, 63, 64, 130, 2240})
      for (int L : {1, 16, 17, 128, 129, 1024, 1025, 5000})
        for (int gap : {0, 1, 6})
          for (int bits = 0; bits < 4; ++bits)
            lrec(3, L, C, io, (bits & 1 ? GDN_FLAG_GATE_LOGITS : 0) | GDN_LREC_COMPLEMENT, gap,
                 gap == 1, bits & 1, bits & 2);
  }
  // the one-minute shapes, and sizes near the integer limits
  qk(1, 106480, 20, 20, 112, GDN_BF16, GDN_NORM_RMS, 3, 0, 0, true, true, false);
  lrec(1, 106480, 2240, GDN_BF16, GDN_LREC_COMPLEMENT, 0, 0, true, true);
  lrec(1, 1000000000, 64, GDN_BF16, 0, 0, 0, true, true);
  lrec(1, 2, 500000000, GDN_FP32, 0, 0, 0, true, true);
  pack(1, 2147483647, 1, 4, GDN_BF16, 0, 0);
  printf("%ld expectations, %d failed\n", g_cases, g_fail);
  return g_fail != 0;
}
