// Host-only stand-ins for the launchers of the block's operators, for the
// sanitizer build of their host code (gdn_block_api.hip): nothing is launched.
// Each checks that what it would touch lies inside the regions that
// block_driver.cpp handed to the entry point, and that the row layout or
// vector width it was given fits every pointer and stride.
#include <stdint.h>
#include <stdio.h>

#include "gdn_block_internal.h"
#include "sanitize_regions.h"

namespace {

struct Region {
  uintptr_t base;
  int64_t bytes;
};
Region g_regions[64];
int g_nregions = 0, g_calls = 0, g_bad = 0;

void bad(const char* what, const void* p, int64_t n) {
  ++g_bad;
  fprintf(stderr, "launch stub: %s at %p (%lld)\n", what, p, (long long)n);
}
void need(const void* p, int64_t bytes, const char* what) {
  if (!p) return;
  const uintptr_t a = reinterpret_cast<uintptr_t>(p);
  for (int i = 0; i < g_nregions; ++i) {
    const Region& r = g_regions[i];
    if (a >= r.base && bytes >= 0 && a + (uintptr_t)bytes <= r.base + (uintptr_t)r.bytes) return;
  }
  bad(what, p, bytes);
}
void aligned(const void* p, int64_t n, const char* what) {
  if (p && reinterpret_cast<uintptr_t>(p) % n) bad(what, p, n);
}
int64_t es_of(int io) { return io == gdn::IO_BF16 ? 2 : 4; }

void rows(const gdn::RowView& x, int B, int L, int64_t width, int V, int io, const char* what) {
  if (!x.p) return;
  need(x.p, ((B - 1) * x.sb + (L - 1) * x.sl + width) * es_of(io), what);
  aligned(x.p, V * es_of(io), what);
  if ((B > 1 && x.sb % V) || (L > 1 && x.sl % V)) bad(what, x.p, x.sl);
}
void shape(const gdn::RowShape& r, int io) {
  const bool widths = io == gdn::IO_BF16 ? r.V == 8 || r.V == 4 || r.V == 2 : r.V == 4 || r.V == 2;
  if (!widths || r.lanes * r.V != r.D || r.group < r.lanes || r.group > 64 ||
      (r.group & (r.group - 1)))
    bad("row shape", nullptr, r.V);
}

}  // namespace

extern "C" void sanitize_reset(void) { g_nregions = g_calls = g_bad = 0; }
extern "C" void sanitize_region(const void* base, int64_t bytes) {
  if (base && g_nregions < 64) g_regions[g_nregions++] = {reinterpret_cast<uintptr_t>(base), bytes};
}
extern "C" int sanitize_calls(void) { return g_calls; }
extern "C" int sanitize_violations(void) { return g_bad; }

namespace gdn {

static hipError_t pack(const PackArgs& a, int io) {
  ++g_calls;
  shape(a.row, io);
  const int64_t n = (int64_t)a.B * a.L * a.H;
  rows(a.x, a.B, a.L, (int64_t)a.H * a.row.D, a.row.V, io, "pack x");
  need(a.v, n * a.row.D, "pack values");
  aligned(a.v, a.row.V, "pack values");
  need(a.scale, n, "pack scale");
  return hipSuccess;
}
hipError_t launch_pack8(const PackArgs& a, int io, hipStream_t) { return pack(a, io); }
hipError_t launch_unpack8(const PackArgs& a, int io, hipStream_t) { return pack(a, io); }

int64_t qk_backward_parts(int64_t tokens) {
  const int64_t n = 2 * ((tokens + 3) / 4);
  return n < 1024 ? n : 1024;
}
static void qk(const QkArgs& a, int io, bool packed) {
  ++g_calls;
  shape(a.row, io);
  if (a.pairs % a.row.V) bad("pairs", nullptr, a.pairs);
  const int64_t tokens = (int64_t)a.B * a.L;
  for (int i = 0; i < 2; ++i) {
    const int64_t n = tokens * a.H[i];
    rows(a.x[i], a.B, a.L, (int64_t)a.H[i] * a.row.D, a.row.V, io, "qk x");
    rows(a.dx[i], a.B, a.L, (int64_t)a.H[i] * a.row.D, a.row.V, io, "qk dx");
    need(a.y[i], n * a.row.D * es_of(io), "qk y");
    aligned(a.y[i], a.row.V * es_of(io), "qk y");
    need(a.v8[i], n * a.row.D, "qk values read");
    need(a.s8[i], n, "qk scales read");
    need(a.v8_out[i], n * a.row.D, "qk values written");
    need(a.s8_out[i], n, "qk scales written");
    aligned(a.v8[i], a.row.V, "qk values read");
    aligned(a.v8_out[i], a.row.V, "qk values written");
    need(a.w[i], a.row.D * 4, "qk weights");
    need(a.dw[i], a.row.D * 4, "qk weight gradients");
    if (packed != (a.v8[i] != nullptr)) bad("qk source", a.v8[i], packed);
    if (a.norm && !packed && !a.x[i].p) bad("qk rows", nullptr, i);
  }
  if (a.pairs) need(a.pos, (a.pos_shared ? (int64_t)a.L : tokens) * a.axes * 4, "qk positions");
  need(a.len, (int64_t)a.B * 4, "qk lengths");
  need(a.part, qk_backward_parts(tokens) * a.row.D * 4, "qk parts");
}
hipError_t launch_qk_forward(const QkArgs& a, int io, bool packed, hipStream_t) {
  qk(a, io, packed);
  return hipSuccess;
}
hipError_t launch_qk_backward(const QkArgs& a, int io, bool packed, hipStream_t) {
  qk(a, io, packed);
  return hipSuccess;
}

static void lrec(const LrecArgs& a, int io, int vec) {
  ++g_calls;
  const int64_t BC = (int64_t)a.B * a.C;
  if (vec != 1 && !(io == IO_BF16 && vec == 2)) bad("lrec vec", nullptr, vec);
  if (a.C % vec || (int64_t)a.strips * 64 * vec < a.C) bad("lrec strips", nullptr, a.strips);
  if ((int64_t)a.chunks * kLrecChunk < a.L) bad("lrec chunks", nullptr, a.chunks);
  rows(RowView{a.x, a.x_sb, a.x_sl}, a.B, a.L, a.C, vec, io, "lrec x");
  rows(RowView{a.z, a.z_sb, a.z_sl}, a.B, a.L, a.C, vec, io, "lrec gate");
  rows(RowView{a.dx, a.dx_sb, a.dx_sl}, a.B, a.L, a.C, vec, io, "lrec dx");
  rows(RowView{a.dz, a.dz_sb, a.dz_sl}, a.B, a.L, a.C, vec, io, "lrec dgate");
  need(a.o, a.L * BC * es_of(io), "lrec o");
  need(a.d_o, a.L * BC * es_of(io), "lrec d_o");
  need(a.h0, BC * 4, "lrec state_in");
  need(a.hT, BC * 4, "lrec state_out");
  need(a.dhT, BC * 4, "lrec d_state_out");
  need(a.dh0, BC * 4, "lrec d_state_in");
  need(a.len, (int64_t)a.B * 4, "lrec lengths");
  need(a.enter, a.chunks * BC * 4, "lrec entering states");
  if (a.chunks > 1) {
    if (!a.ticket || !a.agg || !a.pre) bad("lrec workspace", a.ticket, 0);
    need(a.ticket, a.ws_bytes, "lrec cleared workspace");
    const char* end = reinterpret_cast<const char*>(a.ticket) + a.ws_bytes;
    const int64_t agg = end - reinterpret_cast<const char*>(a.agg);
    const int64_t pre = end - reinterpret_cast<const char*>(a.pre);
    if (agg < a.chunks * BC * 8 || pre < (a.chunks / kLrecGroup) * BC * 4)
      bad("lrec words cleared", a.agg, agg);
    need(a.agg, a.chunks * BC * 8, "lrec maps");
    need(a.pre, (a.chunks / kLrecGroup) * BC * 4, "lrec group states");
    aligned(a.agg, 8, "lrec maps");
  }
}
hipError_t launch_lrec_forward(const LrecArgs& a, int io, int vec, bool states, hipStream_t) {
  lrec(a, io, vec);
  if (states ? !a.enter : !a.o) bad("lrec outputs", a.o, states);
  return hipSuccess;
}
hipError_t launch_lrec_backward(const LrecArgs& a, int io, int vec, hipStream_t) {
  lrec(a, io, vec);
  if (!a.enter || !a.dx || !a.dz) bad("lrec gradients", a.enter, 0);
  return hipSuccess;
}

}  // namespace gdn
