// Threads that ask for a device's value at once, while it is being made (built and run by test_per_device.py).
#include <chrono>
#include <cstdio>
#include <thread>
#include <vector>

#include "per_device.h"

struct Clusters {
    int n[4];
};

int main() {
    static a2av::PerDevice<Clusters> cache;
    std::atomic<int> asked{0}, wrong{0}, refused{0};
    const auto query = [&](Clusters &c) {
        if (asked.fetch_add(1) == 0) return false;  // the first one fails, and is asked again
        for (int i = 0; i < 4; ++i) {
            c.n[i] = 100 + i;
            std::this_thread::sleep_for(std::chrono::milliseconds(5));
        }
        return true;
    };
    std::vector<std::thread> threads;
    for (int t = 0; t < 16; ++t)
        threads.emplace_back([&] {
            for (int dev : {3, 3}) {
                const Clusters *c = cache.get(dev, query);
                if (!c) ++refused;
                else
                    for (int i = 0; i < 4; ++i) wrong += c->n[i] != 100 + i;
            }
        });
    for (auto &t : threads) t.join();
    const bool outside = cache.get(-1, query) || cache.get(64, query);
    std::printf("%d %d %d %d\n", asked.load(), refused.load(), wrong.load(), outside ? 1 : 0);
}
