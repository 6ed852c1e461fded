// Random-input driver of the host side of routing, combining and the 4-bit
// products (csrc/api_route.cpp, csrc/api_affine.cpp, the rules of
// csrc/affine_choice.hpp).  Built with AddressSanitizer and
// UndefinedBehaviorSanitizer by tests/test_sanitize_route_affine_cpu.py; any
// report aborts the run.  There is no device code: the kernel launchers below
// check instead that what reaches them fits a launch and the workspace.
#include <cstdio>
#include <cstdlib>
#include <string>
#include <vector>

#include "../../adapter_lora_segments_amd/csrc/affine_choice.hpp"
#include "../../adapter_lora_segments_amd/csrc/expert_choice.hpp"
#include "../../adapter_lora_segments_amd/csrc/route.hpp"
#include "../../include/mlora.h"

namespace {

uint64_t g_state = 0x9E3779B97F4A7C15ull;
uint64_t next() {  // xorshift64*
  g_state ^= g_state >> 12;
  g_state ^= g_state << 25;
  g_state ^= g_state >> 27;
  return g_state * 0x2545F4914F6CDD1Dull;
}
int64_t uni(int64_t lo, int64_t hi) { return lo + (int64_t)(next() % (uint64_t)(hi - lo + 1)); }
bool chance(int pct) { return uni(0, 99) < pct; }
int64_t spread(int bits) { return uni(0, ((int64_t)1 << uni(0, bits)) - 1); }

std::string g_msg;
long g_launches = 0, g_ok = 0, g_err = 0;
const uintptr_t kWs = uintptr_t(1) << 50;
int64_t g_ws = 0, g_weights = 0;

#define CHECK(x)                                                                    \
  do {                                                                              \
    if (!(x)) {                                                                     \
      std::fprintf(stderr, "%s:%d: %s does not hold\n", __FILE__, __LINE__, #x);    \
      std::abort();                                                                 \
    }                                                                               \
  } while (0)

constexpr int64_t kThreads32 = (int64_t)1 << 32;

char* at(int i) { return reinterpret_cast<char*>((uintptr_t(1) << 40) * (unsigned)(i + 1)); }

}  // namespace

extern "C" {
hipError_t hipGetLastError(void) { return hipSuccess; }
const char* hipGetErrorName(hipError_t) { return "none"; }
const char* hipGetErrorString(hipError_t) { return "none"; }
}

namespace mlora {

void set_last_error(const std::string& m) { g_msg = m; }

static void routed(const RouteArgs& a) {
  ++g_launches;
  CHECK(a.rows > 0 && a.rows < ((int64_t)1 << 31) && a.ld >= a.E && a.E >= 1 && a.E <= MLORA_MAX_EXPERTS && a.k >= 1 && a.k <= 64);
  CHECK(a.k <= a.per_group * a.top_groups || a.n_groups == 1);
  CHECK(a.n_groups >= 1 && a.n_groups <= 64 && a.top_groups >= 1 && (a.n_groups == 1 || a.top_groups < a.n_groups));
  // rows of a workgroup: 64 threads and one row over 1024 experts, else at least four rows of 256
  const int64_t groups = a.E > 1024 ? a.rows : (a.rows + 3) / 4;
  CHECK(groups * (a.E > 1024 ? 64 : 256) < kThreads32);
}
void launch_route(bool, const RouteArgs& a, hipStream_t) {
  routed(a);
  CHECK(a.ids && a.weights && !a.dlogits);
}
void launch_route_backward(bool, const RouteArgs& a, hipStream_t) {
  routed(a);
  CHECK(a.ids && a.dweights && a.dlogits);
}
static void combined(bool f32, const CombineArgs& a) {
  ++g_launches;
  CHECK(a.tokens > 0 && a.k >= 1 && a.k <= 64 && a.tokens * a.k < ((int64_t)1 << 31));
  CHECK(a.d > 0 && a.d % (f32 ? 4 : 8) == 0 && a.limit >= 1);
}
void launch_combine(bool f32, const CombineArgs& a, hipStream_t) {
  combined(f32, a);
  CHECK(a.Y && a.out);
  const int64_t pieces = a.d / (f32 ? 4 : 8);
  int64_t lanes = 1;
  while (lanes < pieces && lanes < 256) lanes *= 2;
  const int64_t per = 256 / lanes, split = (pieces + 255) / 256;
  CHECK((a.tokens + per - 1) / per * split * 256 < kThreads32);
}
void launch_combine_backward(bool f32, const CombineArgs& a, hipStream_t) {
  combined(f32, a);
  CHECK(a.dout && (a.dY || a.dweights) && (!a.dweights || a.Y));
}

void launch_affine_quantize(bool, const void* X, int64_t rows, int64_t cols, int64_t ld, int32_t group, bool,
                            uint8_t* codes, uint32_t* params, void*, hipStream_t) {
  ++g_launches;
  CHECK(X && rows > 0 && cols > 0 && cols % group == 0 && ld >= cols);
  CHECK(rows * (cols / 8) + 255 < ((int64_t)1 << 31));
  CHECK(reinterpret_cast<uint8_t*>(params) - codes == rows * cols / 2);
}
void launch_affine_decode(const uint8_t*, const uint32_t*, int64_t rows, int64_t cols, int32_t, uint16_t* out, hipStream_t) {
  ++g_launches;
  CHECK((rows * (cols / 8) + 255) / 256 <= kMaxGrid && rows * cols == g_weights);
  CHECK(reinterpret_cast<uintptr_t>(out) == kWs && 2 * rows * cols <= g_ws);
}
static void common(const ExpertArgs& a) {
  ++g_launches;
  CHECK(a.rows > 0 && a.N > 0 && a.K > 0 && a.A && a.B && a.C && a.n_experts >= 1 && (a.offsets || a.n_experts == 1));
  CHECK(a.order || (!a.ma.by_order && !a.mc.by_order));
}
void launch_affine_few(const ExpertArgs& a, int32_t group, int rows, int cols, hipStream_t) {
  common(a);
  CHECK(affine_grid(a, rows, cols) <= kMaxGrid && a.K % group == 0 && a.b_expert * a.n_experts * 2 == g_weights);
  CHECK((int64_t)127 * (a.K / 2) + a.K / 2 < ((int64_t)1 << 32));        // offsets within a tile's columns
}
void launch_affine_tile(const ExpertArgs& a, int32_t group, int rows, int parts, hipStream_t) {
  common(a);
  CHECK(affine_grid(a, rows, 128) <= kMaxGrid && a.K % group == 0 && (parts == 1 || parts == 2));
}
void launch_affine_dx(const ExpertArgs& a, int32_t group, int rows, hipStream_t) {
  common(a);
  CHECK(affine_grid(a, rows, 128) <= kMaxGrid && a.N % group == 0);
}
void launch_expert_rows(ExpertForm form, bool b_kc, const ExpertArgs& a, hipStream_t) {
  common(a);
  CHECK(form == ExpertForm::kBf16 && reinterpret_cast<uintptr_t>(a.B) == kWs);
  CHECK(max_row_tiles(a.rows, a.n_experts, 64) * ((a.N + 127) / 128) < ((int64_t)1 << 31));
  const double bytes = 2.0 * a.K * a.N;
  const Choice& c = b_kc ? choose(kBf16Nk, false, a, bytes) : choose(kBf16Kn, false, a, bytes);
  if (c.few) CHECK(rows_grid(a, c.rows, c.cols) <= kMaxGrid);
}

}  // namespace mlora

namespace {

void count(mlora_status st, long before, long launched) {
  if (st == MLORA_OK) {
    ++g_ok;
    CHECK(g_launches == before + launched);
  } else {
    ++g_err;
    CHECK(st < 0 && g_launches == before && !g_msg.empty());
    g_msg.clear();
  }
}
int32_t odd(int32_t v, int pct, int64_t lo, int64_t hi) { return chance(pct) ? (int32_t)uni(lo, hi) : v; }
mlora_dtype dtype() { return (mlora_dtype)odd((int32_t)uni(0, 1), 3, -1, 3); }
int64_t many() { return chance(4) ? std::vector<int64_t>{-1, (int64_t)1 << 31, INT64_MAX, INT64_MIN, (1 << 26) + 8}[uni(0, 4)] : spread(31); }

void routes() {
  const int32_t groups = odd((int32_t)(1 << uni(0, 4)), 3, -1, 70);
  const int32_t E = odd((int32_t)(groups * (1 + spread(8))), 3, -1, 5000);
  mlora_router r{E, odd((int32_t)uni(1, 8), 5, -1, 70), odd((int32_t)uni(0, 1), 2, -1, 3), groups,
                 odd((int32_t)uni(1, groups > 0 ? groups : 1), 3, -1, 70), odd((int32_t)uni(0, 1), 2, -1, 3),
                 odd((int32_t)uni(0, 1), 2, -1, 3), 1.5f};
  const int64_t rows = many(), ld = chance(10) ? spread(13) - 2 : E + uni(0, 3);
  const mlora_dtype dt = dtype();
  const int off = chance(5) ? 1 : 0;
  long before = g_launches;
  count(mlora_route(chance(1) ? nullptr : &r, chance(2) ? nullptr : at(1) + off, dt, rows, ld,
                    reinterpret_cast<float*>(chance(50) ? at(2) : nullptr), reinterpret_cast<int32_t*>(at(3)),
                    reinterpret_cast<float*>(at(4)), nullptr), before, rows > 0);
  before = g_launches;
  count(mlora_route_backward(&r, at(1), dt, rows, ld, reinterpret_cast<int32_t*>(at(3)), reinterpret_cast<float*>(at(4)),
                             chance(2) ? nullptr : at(5) + off, nullptr), before, rows > 0);
}

void combines() {
  const int32_t k = odd((int32_t)uni(1, 8), 5, -1, 70), E = odd((int32_t)spread(8), 3, -4, 0);
  const int64_t tokens = many(), d = chance(5) ? spread(21) - 3 : 8 * spread(13);
  const mlora_dtype dt = dtype();
  auto* ids = reinterpret_cast<int32_t*>(chance(50) ? at(3) : nullptr);
  auto* w = reinterpret_cast<float*>(chance(50) ? at(4) + (chance(3) ? 2 : 0) : nullptr);
  long before = g_launches;
  count(mlora_combine(at(1) + (chance(3) ? 8 : 0), dt, tokens, k, d, ids, E, w, chance(50) ? at(5) : nullptr,
                      chance(2) ? nullptr : at(6), nullptr), before, tokens > 0);
  void* dy = chance(80) ? at(6) : nullptr;
  auto* dw = reinterpret_cast<float*>(chance(50) ? at(7) : nullptr);
  before = g_launches;
  count(mlora_combine_backward(at(5), chance(80) ? at(1) : nullptr, dt, tokens, k, d, ids, E, w, dy, dw, nullptr), before,
        tokens > 0 && (dy || dw));
}

int32_t group_of() { return odd((int32_t)32 << uni(0, 2), 3, -1, 256); }

void quantizes() {
  const int32_t g = group_of();
  const int64_t cols = chance(5) ? spread(21) : (int64_t)g * spread(10), rows = many();
  const int64_t ld = chance(10) ? spread(21) - 4 : cols + 8 * uni(0, 2);
  long before = g_launches;
  count(mlora_affine_quantize(at(1) + (chance(3) ? 4 : 0), dtype(), rows, cols, ld, g, odd((int32_t)uni(0, 1), 2, -1, 3),
                              chance(2) ? nullptr : at(2), chance(50) ? at(3) : nullptr, nullptr), before, rows > 0);
}

void products() {
  const int32_t g = group_of(), k = chance(50) ? 1 : odd((int32_t)uni(1, 8), 5, -1, 70);
  const int32_t xo = odd(k > 1 ? 1 : (int32_t)uni(0, 1), 3, -1, 3), yo = odd((int32_t)uni(0, 1), 3, -1, 3);
  const int32_t E = odd((int32_t)(1 + spread(7)), 3, -1, 5000);
  const int64_t rows = chance(4) ? many() : k * spread(chance(20) ? 27 : 14);
  mlora_affine_shape s{rows, chance(3) ? spread(22) : (int64_t)g * (1 + spread(9)), chance(3) ? spread(22) : 8 * (1 + spread(12)),
                       E, g, k, xo, yo};
  int64_t f = -1, b = -1;
  const long before = g_launches;
  const mlora_status st = mlora_affine_workspace(&s, &f, &b);
  CHECK(g_launches == before);
  if (st != MLORA_OK) {
    CHECK(f == -1 && b == -1);
    f = b = 0;
  } else {
    g_weights = s.d_in * s.d_out * E;
    CHECK((f == 0) == (rows < 1024 * (int64_t)E) && b == f && (f == 0 || f == 2 * g_weights));
    // fewer rows need no more
    mlora_affine_shape less = s;
    less.rows = k * uni(0, rows / k);
    int64_t f2 = 0, b2 = 0;
    CHECK(mlora_affine_workspace(&less, &f2, &b2) == MLORA_OK && f2 <= f && b2 <= b);
  }
  const bool tables = E != 1 || xo || yo || chance(50);
  auto* off = reinterpret_cast<int32_t*>(tables && !chance(2) ? at(3) : nullptr);
  auto* order = reinterpret_cast<int32_t*>(tables && !chance(2) ? at(4) : nullptr);
  for (int back = 0; back < 2; ++back) {
    g_ws = (back ? b : f) - (chance(5) ? 1 : 0);
    if (g_ws < 0) g_ws = 0;
    void* ws = g_ws ? reinterpret_cast<void*>(kWs) : nullptr;
    const bool decoded = (back ? b : f) > 0;
    const long was = g_launches;
    char* y = chance(2) ? nullptr : at(6) + (chance(3) ? 8 : 0);
    count(back ? mlora_affine_backward(&s, at(1), at(2), off, order, y, ws, (size_t)g_ws, nullptr)
               : mlora_affine_forward(&s, at(1), at(2), off, order, y, ws, (size_t)g_ws, nullptr),
          was, rows > 0 ? (decoded ? 2 : 1) : 0);
  }
}

}  // namespace

int main(int argc, char** argv) {
  const long cases = argc > 1 ? std::atol(argv[1]) : 20000;
  g_state ^= argc > 2 ? (uint64_t)std::atoll(argv[2]) * 0x100000001B3ull : 0;
  for (long c = 0; c < cases; ++c) {
    routes();
    combines();
    quantizes();
    products();
  }
  // the quantizer's row of an element: exact over a launch's range
  for (int i = 0; i < 200000; ++i) {
    const int32_t d = (int32_t)(4 + spread(17));
    const mlora::DivBy v = mlora::div_by(d);
    const uint32_t n = (uint32_t)(i < 64 ? 0x7FFFFFFFu - (uint32_t)i : spread(31));
    CHECK((uint32_t)(((uint64_t)n * v.mul) >> 32 >> v.shift) + (v.mul ? 0u : n) == n / (uint32_t)d);
  }
  std::printf("cases %ld: %ld accepted, %ld refused, %ld launches\n", cases, g_ok, g_err, g_launches);
  return 0;
}
