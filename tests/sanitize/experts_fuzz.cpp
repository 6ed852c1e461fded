// Random-input driver of the host side of the grouped expert products, the row
// grouping and the MXFP4 quantizer (csrc/api_experts.cpp, the rules of
// csrc/expert_choice.hpp).  Built with AddressSanitizer and
// UndefinedBehaviorSanitizer by tests/test_sanitize_experts_cpu.py; any report
// aborts the run.  There is no device code: the kernel launchers below check
// instead that what reaches them fits a launch and the caller's workspace.
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <string>
#include <vector>

#include "../../adapter_lora_segments_amd/csrc/expert_choice.hpp"
#include "../../adapter_lora_segments_amd/csrc/kernels.hpp"
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
int64_t spread(int bits) { return uni(0, ((int64_t)1 << uni(0, bits)) - 1); }   // every order of magnitude alike

std::string g_msg;
long g_launches = 0, g_ok = 0, g_err = 0;
const uintptr_t kWs = uintptr_t(1) << 50;      // the caller's workspace, [kWs, kWs + g_ws)
int64_t g_ws = 0;

#define CHECK(x)                                                                    \
  do {                                                                              \
    if (!(x)) {                                                                     \
      std::fprintf(stderr, "%s:%d: %s does not hold\n", __FILE__, __LINE__, #x);    \
      std::abort();                                                                 \
    }                                                                               \
  } while (0)

void in_ws(const void* p, int64_t bytes) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p);
  CHECK(bytes >= 0 && a >= kWs && (int64_t)(a - kWs) <= g_ws - bytes);
}
bool of_ws(const void* p) { return reinterpret_cast<uintptr_t>(p) >= kWs && reinterpret_cast<uintptr_t>(p) < kWs + (uintptr_t(1) << 49); }

}  // namespace

extern "C" {
hipError_t hipGetLastError(void) { return hipSuccess; }
const char* hipGetErrorName(hipError_t) { return "none"; }
const char* hipGetErrorString(hipError_t) { return "none"; }
}

namespace mlora {

void set_last_error(const std::string& m) { g_msg = m; }

void launch_group_rows(const int32_t*, int64_t rows, int32_t n, int32_t*, int32_t*, int32_t* counts, hipStream_t) {
  ++g_launches;
  CHECK(rows >= 0 && rows < ((int64_t)1 << 31) && n >= 1 && n <= MLORA_MAX_EXPERTS);
  if (rows <= kGroupOneLaunch) return;
  const int64_t part = group_part_rows(rows), parts = (rows + part - 1) / part;
  CHECK(parts >= 1 && parts <= kGroupMaxParts && part % 1024 == 0);
  in_ws(counts, 4 * parts * n);
}

void launch_quant_mx4(bool f32, bool down, const void*, int64_t rows, int64_t cols, int64_t ld, uint8_t* codes,
                      uint8_t* scales, void*, hipStream_t) {
  ++g_launches;
  const int64_t wide = f32 ? 64 : 128;
  const int64_t gx = down ? (rows / 32 + 3) / 4 : (rows * (cols / 8) + 255) / 256, gy = down ? (cols + wide - 1) / wide : 1;
  CHECK(gx >= 1 && gy >= 1 && gy <= 65535 && gx * gy * 256 < ((int64_t)1 << 32) && ld >= cols);
  if (of_ws(codes)) {                      // a forward's activations
    in_ws(codes, rows * (cols / 2));
    in_ws(scales, rows * (cols / 32));
    CHECK(scales >= codes + rows * (cols / 2));
  }
}

void launch_dequant_mx4(bool nk, const uint8_t*, const uint8_t*, int64_t d_in, int64_t d_out, uint16_t* out, hipStream_t) {
  ++g_launches;
  CHECK(nk && (d_out * (d_in / 32) + 255) / 256 <= kMaxGrid);
  in_ws(out, 2 * d_in * d_out);
}

template <int N>
static void rules(const Choice (&t)[N], bool fixed, const ExpertArgs& a, double per) {
  const Choice& c = choose(t, fixed, a, per * a.K * a.N);
  if (c.few || fixed) CHECK(rows_grid(a, c.rows, c.cols) <= kMaxGrid);
}
static void common(const ExpertArgs& a) {
  ++g_launches;
  CHECK(a.rows >= 0 && a.n_experts >= 1 && (a.offsets || a.n_experts == 1));
  CHECK(a.order || (!a.ma.by_order && !a.mb.by_order && !a.mc.by_order));
}
void launch_expert_rows(ExpertForm form, bool b_kc, const ExpertArgs& a, hipStream_t) {
  common(a);
  CHECK(a.rows > 0 && a.N > 0 && a.K > 0 && a.A && a.B && a.C);
  // tiles of 64 rows of groups that hold all rows, and along N
  CHECK(max_row_tiles(a.rows, a.n_experts, 64) * ((a.N + 127) / 128) < ((int64_t)1 << 31));
  switch (form) {
    case ExpertForm::kBf16: b_kc ? rules(kBf16Nk, false, a, 2) : rules(kBf16Kn, false, a, 2); break;
    case ExpertForm::kF32: b_kc ? rules(kF32Nk, true, a, 4) : rules(kF32Kn, true, a, 4); break;
    case ExpertForm::kW4A16: rules(kW4A16, false, a, .53125); break;
    case ExpertForm::kW4A4: {
      rules(kW4A4, false, a, .53125);
      CHECK(a.ma.by_order || of_ws(a.A));
      in_ws(a.A, a.K / 2);
      break;
    }
  }
}
void launch_expert_dw(bool f32, const ExpertArgs& a, hipStream_t) {
  common(a);
  CHECK(a.M > 0 && a.N > 0 && a.C && (a.rows == 0 || (a.A && a.B)));
  const int64_t E = a.offsets ? a.n_experts : 1, t = dw_tile(f32, E, a.M, a.N);
  const int64_t tt = ((a.M + t - 1) / t) * ((a.N + t - 1) / t);
  if (a.chunk == 0) {
    CHECK(8 * E * ((tt + 7) / 8) <= kMaxGrid);
    return;
  }
  CHECK(((int64_t)a.rows / a.chunk + E) * tt + 7 <= kMaxGrid && E * ((a.c_expert / 4 + 255) / 256) <= kMaxGrid);
  CHECK(a.c_expert == (int64_t)a.M * a.N && a.c_expert % 4 == 0);
  // slots of the chunks of any groups: two a chunk's rows, and never fewer than one group of all rows needs
  const int64_t slots = 2 * (int64_t)a.rows / a.chunk;
  CHECK(pieces_of(a.rows, a.chunk) <= slots);
  in_ws(a.part, slots * a.c_expert * 4);
}

}  // namespace mlora

namespace {

int64_t dim() {
  if (chance(4)) return std::vector<int64_t>{0, -8, 12, 100, (1 << 20) + 8, INT64_MAX}[uni(0, 5)];
  if (chance(10)) return 1 << 20;
  if (chance(40)) return 128 * (1 + spread(12));
  return 8 * (1 + spread(17));
}
int32_t flag() { return (int32_t)(chance(2) ? uni(-1, 3) : uni(0, 1)); }

mlora_expert_shape make_shape() {
  mlora_expert_shape s{};
  s.top_k = (int32_t)(chance(3) ? uni(-1, 70) : chance(60) ? 1 : uni(1, 64));
  s.x_by_order = s.top_k > 1 && chance(95) ? 1 : flag();
  s.rows = chance(3) ? uni(-2, 0) : chance(5) ? ((int64_t)1 << 31) - uni(0, 600) : spread(31);
  if (s.top_k > 1 && chance(95)) s.rows = s.rows / s.top_k * s.top_k;
  s.d_in = dim();
  s.d_out = dim();
  s.n_experts = (int32_t)(chance(3) ? uni(-1, 4097) : 1 + spread(12));
  s.dtype = (int32_t)(chance(2) ? uni(-1, 3) : uni(0, 1));
  s.w_layout = (int32_t)(chance(2) ? uni(-1, 3) : uni(0, 1));
  if (chance(40)) {
    s.w_format = 2, s.dtype = 1, s.w_layout = 1;
    s.act_format = chance(50) ? 2 : 0;
  } else if (chance(2)) {
    s.w_format = (int32_t)uni(-1, 3), s.act_format = (int32_t)uni(-1, 3);
  }
  s.y_by_order = flag();
  s.grad_accumulate = flag();
  return s;
}

void expect_error(mlora_status s) {
  CHECK(s < 0 && !g_msg.empty());
  g_msg.clear();
}

char* at(int i) { return reinterpret_cast<char*>((uintptr_t(1) << 40) + ((uintptr_t)i << 36)); }

void products() {
  const mlora_expert_shape most = make_shape();
  int64_t both = -7, fwd = -7;
  const mlora_status st = mlora_expert_workspace(&most, &both);
  CHECK(mlora_expert_forward_workspace(&most, &fwd) == st);
  char* ws = reinterpret_cast<char*>(kWs);
  int32_t* off = reinterpret_cast<int32_t*>(at(1));
  int32_t* ord = reinterpret_cast<int32_t*>(at(2));
  float* dW = reinterpret_cast<float*>(at(8));
  if (st != MLORA_OK) {
    ++g_err;
    CHECK(both == -7 && fwd == -7);
    g_ws = (int64_t)1 << 49;
    const long before = g_launches;
    expect_error(mlora_expert_forward(&most, at(3), at(4), off, ord, at(5), ws, (size_t)g_ws, nullptr));
    expect_error(mlora_expert_backward(&most, at(6), at(3), at(4), off, ord, at(7), dW, ws, (size_t)g_ws, nullptr));
    CHECK(g_launches == before);
    return;
  }
  ++g_ok;
  CHECK(both >= fwd && fwd >= 0);
  // a call of as many rows, or fewer, with exactly the reported workspace
  mlora_expert_shape s = most;
  if (chance(60)) s.rows = uni(0, most.rows) / most.top_k * most.top_k;
  g_ws = fwd;
  CHECK(mlora_expert_forward(&s, at(3), at(4), off, ord, at(5), ws, (size_t)fwd, nullptr) == MLORA_OK);
  g_ws = both;
  const bool w4 = s.w_format == MLORA_W0_MXFP4;
  CHECK(mlora_expert_backward(&s, at(6), at(3), at(4), off, ord, at(7), w4 ? nullptr : dW, ws, (size_t)both, nullptr) ==
        MLORA_OK);
  // damaged ones
  const long before = g_launches;
  if (s.rows > 0) {
    int64_t need = -1;
    CHECK(mlora_expert_forward_workspace(&s, &need) == MLORA_OK && need <= fwd);
    if (need > 0) {
      expect_error(mlora_expert_forward(&s, at(3), at(4), off, ord, at(5), ws, (size_t)need - 1, nullptr));
      expect_error(mlora_expert_forward(&s, at(3), at(4), off, ord, at(5), nullptr, (size_t)need, nullptr));
      expect_error(mlora_expert_forward(&s, at(3), at(4), off, ord, at(5), ws + 4, (size_t)need, nullptr));
    }
    expect_error(mlora_expert_forward(&s, nullptr, at(4), off, ord, at(5), ws, (size_t)fwd, nullptr));
    expect_error(mlora_expert_forward(&s, at(3), at(4), off, ord, at(5) + 8, ws, (size_t)fwd, nullptr));
    expect_error(mlora_expert_backward(&s, nullptr, at(3), at(4), off, ord, at(7), nullptr, ws, (size_t)both, nullptr));
    expect_error(mlora_expert_backward(&s, at(6), at(3), nullptr, off, ord, at(7), nullptr, ws, (size_t)both, nullptr));
    if (w4)
      expect_error(mlora_expert_backward(&s, at(6), nullptr, at(4), off, ord, at(7), nullptr, ws,
                                         (size_t)(2 * s.n_experts * s.d_in * s.d_out - 1), nullptr));
  }
  if (w4) expect_error(mlora_expert_backward(&s, at(6), at(3), at(4), off, ord, at(7), dW, ws, (size_t)both, nullptr));
  if (s.n_experts > 1)
    expect_error(mlora_expert_forward(&s, at(3), at(4), nullptr, ord, at(5), ws, (size_t)fwd, nullptr));
  if (s.x_by_order || s.y_by_order)
    expect_error(mlora_expert_forward(&s, at(3), at(4), off, nullptr, at(5), ws, (size_t)fwd, nullptr));
  CHECK(g_launches == before);
}

void grouping() {
  const int64_t rows = chance(5) ? uni(-2, 0) : chance(5) ? ((int64_t)1 << 31) - uni(0, 3) : spread(31);
  const int32_t n = (int32_t)(chance(4) ? uni(-1, 4098) : 1 + spread(12));
  int64_t need = -7;
  const mlora_status st = mlora_group_rows_workspace(rows, n, &need);
  int32_t* ids = reinterpret_cast<int32_t*>(at(1));
  int32_t* off = reinterpret_cast<int32_t*>(at(2));
  int32_t* ord = reinterpret_cast<int32_t*>(at(3));
  char* ws = reinterpret_cast<char*>(kWs);
  g_ws = st == MLORA_OK ? need : 0;
  if (st != MLORA_OK) {
    ++g_err;
    CHECK(need == -7);
    expect_error(mlora_group_rows(ids, rows, n, off, ord, ws, (size_t)1 << 40, nullptr));
    return;
  }
  ++g_ok;
  const int64_t fewer = chance(50) ? rows : uni(0, rows);
  CHECK(mlora_group_rows(ids, fewer, n, off, ord, ws, (size_t)need, nullptr) == MLORA_OK);
  if (need > 0) expect_error(mlora_group_rows(ids, rows, n, off, ord, ws, (size_t)need - 1, nullptr));
  expect_error(mlora_group_rows(ids, rows, n, nullptr, ord, ws, (size_t)need, nullptr));
}

void quantizer() {
  const int64_t rows = chance(5) ? uni(-33, 0) : spread(31), cols = dim();
  const int32_t down = flag();
  const int64_t r = down == 1 && chance(90) ? rows / 32 * 32 : rows;
  const int64_t ld = chance(10) ? uni(-8, 1 << 20) : cols < (1 << 30) ? cols + 8 * uni(0, 3) : cols;
  const mlora_dtype dt = (mlora_dtype)(chance(3) ? uni(-1, 3) : uni(0, 1));
  g_ws = 0;
  const long before = g_launches;
  const mlora_status st = mlora_microscale_quantize(at(1), dt, r, cols, ld, down, at(2), chance(50) ? at(3) : nullptr, nullptr);
  if (st == MLORA_OK) {
    ++g_ok;
    CHECK(g_launches == before + (r > 0 ? 1 : 0));
    if (r > 0) expect_error(mlora_microscale_quantize(at(1) + 4, dt, r, cols, ld, down, at(2), nullptr, nullptr));
  } else {
    ++g_err;
    CHECK(g_launches == before);
    expect_error(st);
  }
}

}  // namespace

int main(int argc, char** argv) {
  const long cases = argc > 1 ? std::atol(argv[1]) : 20000;
  g_state ^= argc > 2 ? (uint64_t)std::atoll(argv[2]) * 0x100000001B3ull : 0;
  for (long c = 0; c < cases; ++c) {
    products();
    grouping();
    quantizer();
  }
  // the divisor of top_k: exact over the whole range of rows
  for (int32_t d = 1; d <= 64; ++d) {
    const mlora::DivBy v = mlora::div_by(d);
    for (int i = 0; i < 4000; ++i) {
      const uint32_t n = (uint32_t)(i < 64 ? 0x7FFFFFFFu - (uint32_t)i : spread(31));
      const uint32_t q = (uint32_t)(((uint64_t)n * v.mul) >> 32 >> v.shift) + (v.mul ? 0u : n);
      CHECK(q == n / (uint32_t)d);
    }
  }
  std::printf("cases %ld: %ld accepted, %ld refused, %ld launches\n", cases, g_ok, g_err, g_launches);
  return 0;
}
