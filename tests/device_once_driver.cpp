// Prints how often csrc/device_once.h ran a set-up for each of a line of devices ("device calls" a line), the first call on device 3 failing.
#include <cstdio>

#include "device_once.h"

int main() {
  static detattn::DeviceOnce once, other;
  int calls[70] = {};
  const int order[] = {0, 0, 1, 0, 1, 63, 63, 3, 3, 3, 64, 64, -1};
  for (int d : order) {
    const int e = once(d, [&] { return ++calls[d < 0 ? 69 : d] == 1 && d == 3 ? 7 : 0; });
    if (e != 0) std::printf("failed %d %d\n", d, e);
  }
  const int shown[] = {0, 1, 3, 63, 64, 69};
  for (int d : shown) std::printf("%d %d\n", d, calls[d]);
  int more = 0;
  other(0, [&] { return more++; });
  std::printf("other %d\n", more);
}
