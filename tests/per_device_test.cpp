// csrc/per_device.h against a runtime of two devices that counts what it is asked (test code).
#include "per_device.h"

#include <cstdio>

static int device = 0, asked = 0;
static cudaError_t answer = cudaSuccess;
extern "C" cudaError_t cudaGetDevice(int *dev) {
  *dev = device;
  return device < 0 ? cudaErrorNoDevice : cudaSuccess;
}

static void f(int) {}
static void g(int) {}

#define CHECK(x)                                  \
  if (!(x)) {                                     \
    std::printf("line %d: %s\n", __LINE__, #x);   \
    return 1;                                     \
  }

int main() {
  auto ask = [](ssd::PerDevice &p, int truth) {
    int v = -1;
    const cudaError_t e = p.get(v, [&](int &out) {
      ++asked;
      out = truth;
      return answer;
    });
    return e == cudaSuccess ? v : -2;
  };
  ssd::PerDevice &f4 = ssd::clusters_held<f, 17>(4), &f5 = ssd::clusters_held<f, 17>(5), &g4 = ssd::clusters_held<g, 17>(4);
  CHECK(&f4 != &f5 && &f4 != &g4 && &f4 == &(ssd::clusters_held<f, 17>(4)));
  CHECK(ask(f4, 7) == 7 && asked == 1);
  CHECK(ask(f4, 9) == 7 && asked == 1);                    // kept
  CHECK(ask(g4, 9) == 9 && ask(f5, 0) == 0 && asked == 3);  // another kernel of the same type, another size
  CHECK(ask(f5, 1) == 0 && asked == 3);                    // 0 is an answer
  device = 1;
  CHECK(ask(f4, 5) == 5 && asked == 4);  // another device
  device = 0;
  CHECK(ask(f4, 9) == 7 && asked == 4);
  device = 64;  // past the table: asked each time
  CHECK(ask(f4, 3) == 3 && ask(f4, 4) == 4 && asked == 6);
  device = 2;
  answer = cudaErrorInvalidValue;
  CHECK(ask(f4, 3) == -2 && asked == 7);  // an error is not kept
  answer = cudaSuccess;
  CHECK(ask(f4, 6) == 6 && asked == 8);
  device = -1;
  CHECK(ask(f4, 6) == -2 && asked == 8);
  return 0;
}
